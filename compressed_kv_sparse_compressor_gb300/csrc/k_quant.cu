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

#include <climits>

#include <cuda_bf16.h>

namespace ds4c {

namespace {

// Two floats in a 64-bit register: sm_103a adds, multiplies and fuses both in one issue slot.
using F2 = uint64_t;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// a - b, rounded once (the product with -1 is exact)
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, f2(-1.f, -1.f), a); }

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
// The same for the pair's squares, 0 <= v^2 <= s: the rounded sum t = s + v^2, whose step t - s is exact
// (Dekker, 1971), and what the step lacks to v^2 in one fused product.
__device__ __forceinline__ void add_square(F2 &s, F2 &c, F2 v) {
    const F2 t = fma2(v, v, s);
    c = add2(c, fma2(v, v, sub2(s, t)));
    s = t;
}

// Sum of (s, c) pairs over a row's threads (blockDim.x), the same value in each.  sm: 2 * 32 floats.
__device__ __forceinline__ void row_sum(float &s, float &c, float *sm) {
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

// (v + lo)^-1/2 as r + r e / 2: CUDA's rsqrtf, then the series of (1 - e)^-1/2
// in the residual e = 1 - (v + lo) r^2, which two fused products give exactly enough.
__device__ __forceinline__ float rsqrt_pair(float v, float lo, float &half_e) {
    const float r = rsqrtf(v);
    const float t = __fmul_rn(r, r), tl = fmaf(r, r, -t);
    float e = fmaf(-v, t, 1.f);
    e = __fsub_rn(e, fmaf(v, tl, __fmul_rn(lo, t)));
    half_e = 0.5f * fmaf(0.75f * e, e, e);
    return r;
}

// ((s + c) / d + eps)^-1/2 rounded once to float, 1 / d as a sum of two floats.  DOWN: times 2^-80, where the result may
// be subnormal: in 64 bits up to that one rounding.
template <bool DOWN>
__device__ __forceinline__ float rstd_of(float s, float c, float inv_d, float inv_d_lo, float eps) {
    const float ph = __fmul_rn(s, inv_d);
    float lo = fmaf(s, inv_d, -ph);
    lo = fmaf(s, inv_d_lo, lo);
    lo = fmaf(c, inv_d, lo);
    float v = ph;
    add_exact(v, lo, eps);
    const float vn = __fadd_rn(v, lo);
    float half_e;
    const float r = rsqrt_pair(vn, __fsub_rn(lo, __fsub_rn(vn, v)), half_e);
    return DOWN ? __double2float_rn(fma((double)r, (double)half_e, (double)r) * 0x1p-80) : fmaf(r, half_e, r);
}

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.f;
}
// Largest of m, |a| and |b|; NaN if one is NaN.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
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

// Codes of two values (the lower byte a's); NaN gives the NaN code.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float nan_unless_finite(float v) { return fabsf(v) < INFINITY ? v : NAN; }
// Codes of 8 values at the inverse scale; FINITE: none is infinite (an infinity would saturate).
template <bool FINITE>
__device__ __forceinline__ uint2 codes(const F2 (&y)[4], float inv) {
    uint32_t w[4];
    const F2 inv2 = f2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float2 v = unpack(mul2(y[i], inv2));
        if (!FINITE) v.x = nan_unless_finite(v.x), v.y = nan_unless_finite(v.y);
        w[i] = codes2(v.x, v.y);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A thread's 8 values of a 128-block group.  VEC: 8 consecutive ones (base is a multiple of 8, d too,
// everything aligned), 16 lanes to a block of 128.  Otherwise the warp's 256 values lie lane by
// lane: value j of the thread is at base + 32 j, so that single accesses are coalesced whatever the
// rows' alignment, and values 0-3 and 4-7 belong to two blocks of 128 over all 32 lanes.
template <bool VEC>
__device__ __forceinline__ int first_of(int i) {
    const int t = threadIdx.x;
    return VEC ? (i * (int)blockDim.x + t) * 8 : i * (int)blockDim.x * 8 + t / 32 * 256 + t % 32;
}
// 8 values as they are stored: bf16 pairs in words, floats in pairs.
struct Bf16x8 { uint32_t w[4]; };
struct F32x8 { F2 v[4]; };
template <typename T> struct Held;
template <> struct Held<float> { using type = F32x8; };
template <> struct Held<__nv_bfloat16> { using type = Bf16x8; };

// 16 bytes that are read once.  Volatile: the compiler must not move a load of what the previous
// kernel wrote above the wait for it.
__device__ __forceinline__ uint4 load16(const void *p) {
    uint4 v;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ F2 f2(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int base, int d, F32x8 &h) {
    if (VEC) {
        const uint4 a = load16(p + base), b = load16(p + base + 4);
        h.v[0] = f2(a.x, a.y), h.v[1] = f2(a.z, a.w), h.v[2] = f2(b.x, b.y), h.v[3] = f2(b.z, b.w);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = base + 32 * i < d ? p[base + 32 * i] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) h.v[i] = f2(f[2 * i], f[2 * i + 1]);
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int base, int d, Bf16x8 &h) {
    if (VEC) {
        const uint4 a = load16(p + base);
        h.w[0] = a.x, h.w[1] = a.y, h.w[2] = a.z, h.w[3] = a.w;
    } else {
        uint32_t f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = base + 32 * i < d ? reinterpret_cast<const uint16_t *>(p)[base + 32 * i] : 0u;
#pragma unroll
        for (int i = 0; i < 4; i++) h.w[i] = f[2 * i] | f[2 * i + 1] << 16;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int base, int d, const F32x8 &h) {
    if (VEC) {
        const float2 a = unpack(h.v[0]), b = unpack(h.v[1]), c = unpack(h.v[2]), e = unpack(h.v[3]);
        reinterpret_cast<float4 *>(p + base)[0] = make_float4(a.x, a.y, b.x, b.y);
        reinterpret_cast<float4 *>(p + base)[1] = make_float4(c.x, c.y, e.x, e.y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (base + 32 * i < d) p[base + 32 * i] = i % 2 ? unpack(h.v[i / 2]).y : unpack(h.v[i / 2]).x;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int base, int d, const Bf16x8 &h) {
    if (VEC) {
        *reinterpret_cast<uint4 *>(p + base) = make_uint4(h.w[0], h.w[1], h.w[2], h.w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (base + 32 * i < d) reinterpret_cast<uint16_t *>(p)[base + 32 * i] = (uint16_t)(h.w[i / 2] >> (16 * (i % 2)));
    }
}
// h + r rounded to the type.  Of two bf16 values the float sum is exact or lies too near the larger
// one to reach a bf16 midpoint, so rounding it again gives what one rounding to bf16 gives.
__device__ __forceinline__ void add8(F32x8 &h, const F32x8 &r) {
#pragma unroll
    for (int i = 0; i < 4; i++) h.v[i] = add2(h.v[i], r.v[i]);
}
__device__ __forceinline__ void add8(Bf16x8 &h, const Bf16x8 &r) {
#pragma unroll
    for (int i = 0; i < 4; i++) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(h.w[i]) : "r"(r.w[i]));
}
__device__ __forceinline__ void zero8(F32x8 &h) { h.v[0] = h.v[1] = h.v[2] = h.v[3] = 0; }
__device__ __forceinline__ void zero8(Bf16x8 &h) { h.w[0] = h.w[1] = h.w[2] = h.w[3] = 0; }
__device__ __forceinline__ F2 pair_of(const F32x8 &h, int i) { return h.v[i]; }
__device__ __forceinline__ F2 pair_of(const Bf16x8 &h, int i) {
    return f2(__uint_as_float(h.w[i] << 16), __uint_as_float(h.w[i] & 0xffff0000u));
}
__device__ __forceinline__ void round8(const F2 (&y)[4], F32x8 &h) {
#pragma unroll
    for (int i = 0; i < 4; i++) h.v[i] = y[i];
}
__device__ __forceinline__ void round8(const F2 (&y)[4], Bf16x8 &h) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = unpack(y[i]);
        const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
        h.w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
}

// Scale bytes and codes of a thread's 8 values (every lane of the warp calls this; lanes past d
// hold zeros): the block's maximum over its lanes, NaN or infinite if the block holds such a value,
// then once more over the finite ones (the whole warp together).
template <bool VEC>
__device__ __forceinline__ void quantise8(const F2 (&y)[4], int base, int d, uint8_t *q, uint8_t *scale) {
    float m[2] = {0.f, 0.f};                             // VEC: one block; else one for each half
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 v = unpack(y[i]);
        m[!VEC && i >= 2] = max_abs(m[!VEC && i >= 2], v.x, v.y);
    }
    bool finite = m[0] < INFINITY && m[1] < INFINITY;
    finite = __all_sync(0xffffffffu, finite);
    if (!finite) {
        m[0] = m[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 v = unpack(y[i]);
            m[!VEC && i >= 2] = fmaxf(m[!VEC && i >= 2], fmaxf(finite_abs(v.x), finite_abs(v.y)));
        }
    }
    // over the block's lanes; magnitudes are ordered as integers.  VEC: each half warp's lanes with zeros
    // from the other half
    const uint32_t u0 = __float_as_uint(m[0]), u1 = __float_as_uint(m[1]);
    const bool upper = threadIdx.x % 32 >= 16;
    const uint32_t r0 = __reduce_max_sync(0xffffffffu, VEC && upper ? 0u : u0);
    const uint32_t r1 = __reduce_max_sync(0xffffffffu, VEC ? (upper ? u0 : 0u) : u1);
    m[0] = __uint_as_float(VEC && upper ? r1 : r0);
    m[1] = __uint_as_float(r1);
    const int b0 = scale_byte(m[0]);
    if (VEC) {
        if (base >= d) return;
        const float inv = inverse_scale(b0);
        // rows start on 16 bytes and base is a multiple of 8
        *reinterpret_cast<uint2 *>(q + base) = finite ? codes<true>(y, inv) : codes<false>(y, inv);
        if (threadIdx.x % 16 == 0) scale[base / 128] = (uint8_t)b0;
    } else {
        const int b1 = scale_byte(m[1]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 v = unpack(y[i / 2]);
            const float f = nan_unless_finite((i % 2 ? v.y : v.x) * inverse_scale(i < 4 ? b0 : b1));
            if (base + 32 * i < d) q[base + 32 * i] = (uint8_t)codes2(f, 0.f);
        }
        if (threadIdx.x % 32 == 0) {
            if (base < d) scale[base / 128] = (uint8_t)b0;
            if (base + 128 < d) scale[base / 128 + 1] = (uint8_t)b1;
        }
    }
}

// Largest magnitude of a thread's values, NaN if one is NaN.  bf16 magnitudes are ordered as 16-bit
// integers, NaN above infinity: two at a time.
template <int NI>
__device__ __forceinline__ float largest(const Bf16x8 (&h)[NI]) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 4; j += 2) u = __vimax3_u16x2(u, h[i].w[j] & 0x7fff7fffu, h[i].w[j + 1] & 0x7fff7fffu);
    return __uint_as_float(max(u << 16, u & 0xffff0000u));
}
template <int NI>
__device__ __forceinline__ float largest(const F32x8 (&h)[NI]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 v = unpack(h[i].v[j]);
            m = max_abs(m, v.x, v.y);
        }
    return m;
}

// (s, c) = sum of the squares of h * f, f a power of two.  Each half of the running pair starts at
// the thread's largest square, which makes every term the smaller one of its addition.
template <int NI, typename H>
__device__ __forceinline__ void sum_squares(const H (&h)[NI], float f, float &s, float &c) {
    const float m = largest(h) * f;
    const float top = __fmul_rn(m, m);
    if (!(top < INFINITY)) {                             // an infinity, NaN, or a square past float's range
        s = top;
        c = 0.f;
        return;
    }
    F2 s2 = f2(top, top), c2 = 0;
    const F2 ff = f2(f, f);
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) add_square(s2, c2, f == 1.f ? pair_of(h[i], j) : mul2(pair_of(h[i], j), ff));
    const float2 sv = unpack(s2), cv = unpack(c2);
    s = sv.x;
    c = __fadd_rn(cv.x, cv.y);
    add_exact(s, c, -top);
    add_exact(s, c, sv.y);
    add_exact(s, c, -top);
}

struct NormParams {
    int n, d;
    float eps, inv_d, inv_d_lo;      // inv_d + inv_d_lo = 1 / d
    const void *x, *residual;
    void *residual_out, *y_out;
    int64_t x_ld, residual_ld, residual_out_ld, y_ld, q_ld, scale_ld;
    const float *gain;
    uint8_t *q, *scale;
};

// blockDim.x threads per row (up to NI * 8 values each), blockDim.y rows per block (above one only
// where a row is one warp's).  The row is held as it is stored (a bf16 value in half a register), so
// that a thread can take many values and the fixed work per thread, the meeting of the sums, is spread
// over them.  MAXT: the most threads per block.  INNER: only the last group's places may lie past d (with
// one group, none), so that the others' loads hang on no comparison (16384 x 7168 131 -> 127 us, 4096
// unaligned rows of 4101 45 -> 37).  Many rows are bound by HBM and by how many of them an SM has in flight
// (16384 x 7168 127 us, 95 % of the copy rate: 54 registers hold 5 blocks of 224 threads; 141 us with 4; blocks
// that stay and copy their next row to shared memory beside this one 142 to 163).
template <typename T, int NI, bool VEC, int MAXT, bool INNER>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 4 : 1) rmsnorm_quant_kernel(NormParams p) {
    using H = typename Held<T>::type;
    __shared__ float sm[64];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.n) return;                              // a whole warp: rows of one block are warps then
    // what the places of group i are compared with
    auto end = [&](int i) { return INNER && (i < NI - 1 || NI == 1) ? INT_MAX : p.d; };
    const T *x = static_cast<const T *>(p.x) + row * p.x_ld;
    H h[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int base = first_of<VEC>(i), d = end(i);
        zero8(h[i]);
        if (base < d) load8<VEC>(x, base, d, h[i]);
    }
    if (p.residual) {
        const T *rp = static_cast<const T *>(p.residual) + row * p.residual_ld;
        H r[NI];
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int base = first_of<VEC>(i), d = end(i);
            zero8(r[i]);
            if (base < d) load8<VEC>(rp, base, d, r[i]);
        }
#pragma unroll
        for (int i = 0; i < NI; i++) add8(h[i], r[i]);
    }
    if (p.residual_out) {
        T *o = static_cast<T *>(p.residual_out) + row * p.residual_out_ld;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int base = first_of<VEC>(i), d = end(i);
            if (base < d) store8<VEC>(o, base, d, h[i]);
        }
    }
    if (!p.q && !p.y_out) return;

    float s, c;
    sum_squares(h, 1.f, s, c);
    row_sum(s, c, sm);
    float rstd;
    if (s < 0x1p90f) {
        rstd = rstd_of<false>(s, c, p.inv_d, p.inv_d_lo, p.eps);
    } else {
        // squares near the end of float's range or past it (elements above about 1e13, infinities,
        // NaN): the sum of (h * 2^-80)^2, in which eps vanishes, and 2^-80 put back
        if (blockDim.x > 32) __syncthreads();
        sum_squares(h, 0x1p-80f, s, c);
        row_sum(s, c, sm);
        rstd = s < INFINITY ? rstd_of<true>(s, c, p.inv_d, p.inv_d_lo, 0.f) : s > 0.f ? 0.f : s;
    }

    const F2 rstd2 = f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int base = first_of<VEC>(i), d = end(i);
        F2 y[4];
#pragma unroll
        for (int j = 0; j < 4; j++) y[j] = mul2(pair_of(h[i], j), rstd2);
        if (base < d) {
            if (p.gain) {
                F32x8 g;
                if (VEC) {
                    const float4 a = reinterpret_cast<const float4 *>(p.gain + base)[0];
                    const float4 b = reinterpret_cast<const float4 *>(p.gain + base)[1];
                    g.v[0] = f2(a.x, a.y), g.v[1] = f2(a.z, a.w), g.v[2] = f2(b.x, b.y), g.v[3] = f2(b.z, b.w);
                } else {
                    load8<false>(p.gain, base, d, g);
                }
#pragma unroll
                for (int j = 0; j < 4; j++) y[j] = mul2(y[j], g.v[j]);
            }
            if (p.y_out) {
                H t;
                round8(y, t);
                store8<VEC>(static_cast<T *>(p.y_out) + row * p.y_ld, base, d, t);
            }
        }
        if (p.q) {
            // places past d hold 0 * rstd: zeros, but NaN in a row that is NaN throughout
            if (!(rstd < INFINITY)) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 v = unpack(y[j]);
                    const int step = VEC ? 1 : 32, b = base + 2 * j * step;
                    y[j] = f2(b < d ? v.x : 0.f, b + step < d ? v.y : 0.f);
                }
            }
            quantise8<VEC>(y, base, d, p.q + row * p.q_ld, p.scale + row * p.scale_ld);
        }
    }
}

// One block of 256 threads per 128 x 128 block of weights, 64 values in each thread: VEC a row's
// 128 values in 16 threads, otherwise 4 single ones in each of 32 lanes (two rows per step).
// WHOLE: nothing of the block lies past n or k, so that no load hangs on a comparison (8192 x 8192 floats 52 us,
// 95 % of the copy rate; 60 with the comparisons).
template <typename T, bool VEC, bool WHOLE>
__device__ __forceinline__ void quant_block(int n, int k, const T *w, int64_t w_ld, uint8_t *q, int64_t q_ld, uint8_t *scale,
                                            int64_t scale_ld, float *sm) {
    using H = typename Held<T>::type;
    if (WHOLE) n = k = INT_MAX;
    const int t = threadIdx.x;
    const int base = blockIdx.x * 128 + (VEC ? t % 16 * 8 : t % 32);
    const int row0 = blockIdx.y * 128 + (VEC ? t / 16 : t / 32 * 2);
    // step i, VEC: row row0 + 16 i; else values 0-3 of row row0 + 16 i, 4-7 of the next
    H h[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = row0 + 16 * i;
        zero8(h[i]);
        if (VEC) {
            if (r < n && base < k) load8<true>(w + r * w_ld, base, k, h[i]);
        } else {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                f[j] = r + j / 4 < n && base + 32 * (j % 4) < k ? (float)w[(r + j / 4) * w_ld + base + 32 * (j % 4)] : 0.f;
            const F2 y[4] = {f2(f[0], f[1]), f2(f[2], f[3]), f2(f[4], f[5]), f2(f[6], f[7])};
            round8(y, h[i]);                             // exact: the values are of the type
        }
    }
    float amax = largest(h);
    const bool finite = __syncthreads_and(amax < INFINITY);
    if (!finite) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 a = unpack(pair_of(h[i], j));
                amax = fmaxf(amax, fmaxf(finite_abs(a.x), finite_abs(a.y)));
            }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (t % 32 == 0) sm[t / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) amax = fmaxf(amax, sm[i]);
    const int byte = scale_byte(amax);
    const float inv = inverse_scale(byte);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = row0 + 16 * i;
        const F2 y[4] = {pair_of(h[i], 0), pair_of(h[i], 1), pair_of(h[i], 2), pair_of(h[i], 3)};
        const uint2 c = finite ? codes<true>(y, inv) : codes<false>(y, inv);
        if (VEC) {
            if (r < n && base < k) *reinterpret_cast<uint2 *>(q + r * q_ld + base) = c;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (r + j / 4 < n && base + 32 * (j % 4) < k)
                    q[(r + j / 4) * q_ld + base + 32 * (j % 4)] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j % 4)));
        }
    }
    if (t == 0) scale[blockIdx.y * scale_ld + blockIdx.x] = (uint8_t)byte;
}

// Two blocks to an SM for single loads: with the registers of four the compiler waits for some before it
// makes the next (1000 x 1541 bf16 3.6 us, with four 9.7).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, VEC ? sizeof(T) == 2 ? 4 : 3 : 2)
quant_weight_kernel(int n, int k, const T *w, int64_t w_ld, uint8_t *q, int64_t q_ld, uint8_t *scale, int64_t scale_ld) {
    __shared__ float sm[8];
    pdl_wait();
    pdl_launch_dependents();
    if ((blockIdx.x + 1) * 128 <= k && (blockIdx.y + 1) * 128 <= n)
        quant_block<T, VEC, true>(n, k, w, w_ld, q, q_ld, scale, scale_ld, sm);
    else
        quant_block<T, VEC, false>(n, k, w, w_ld, q, q_ld, scale, scale_ld, sm);
}

// Threads that hold a row in ni groups, and the places that its groups but the last cover (one group: all of it).
int threads_of(int d, int ni) { return (((d + 7) / 8 + ni - 1) / ni + 31) / 32 * 32; }
int inner_end(int ni, int threads) { return (ni == 1 ? threads : (ni - 1) * threads) * 8; }

template <typename T, int NI, int MAXT>
cudaError_t launch_norm(const NormParams &p, bool vec, int threads, cudaStream_t s) {
    // rows of one warp: four to a block
    const int rows = threads == 32 && p.n > 4 ? 4 : 1;
    const dim3 grid((unsigned)((p.n + rows - 1) / rows)), block(threads, rows);
    const bool inner = p.d >= inner_end(NI, threads);
    if (vec && inner) return launch_pdl(rmsnorm_quant_kernel<T, NI, true, MAXT, true>, grid, block, 0, s, p);
    if (vec) return launch_pdl(rmsnorm_quant_kernel<T, NI, true, MAXT, false>, grid, block, 0, s, p);
    if (inner) return launch_pdl(rmsnorm_quant_kernel<T, NI, false, MAXT, true>, grid, block, 0, s, p);
    return launch_pdl(rmsnorm_quant_kernel<T, NI, false, MAXT, false>, grid, block, 0, s, p);
}

// Threads per row.  Few rows: one group of 8 values in each thread, the shortest chain (a row of 4096
// bf16 values in 2.4 us).  Many rows: as few warps as hold the row in 2 groups of each thread, 4 for
// bf16 rows, which are half as wide (4096 x 4096: 25.5 us; 26.8 with 2 groups, 33.5 with 8; 16384 x
// 7168: 131, 195, 170, before INNER; 16384 x 1024 floats: 38 with 2, 42 with 4; 4096 unaligned rows of 4101: 32.6
// with 4, 37 with 2), unaligned ones where that leaves the groups but the last whole (8000 rows of 515: 14.4 with
// 2, 18.5 with 4).
template <typename T>
cudaError_t launch_norm_t(const NormParams &p, bool vec, cudaStream_t s) {
    const int most = sizeof(T) == 2 ? 4 : 2, groups = (p.d + 7) / 8;
    int ni = 1;
    while (ni < most && groups > (p.n >= 512 ? 32 : 1024) * ni && (vec || p.d >= inner_end(2 * ni, threads_of(p.d, 2 * ni)))) ni *= 2;
    while (groups > 1024 * ni) ni *= 2;                  // d = 32768 is 4 groups in each of 1024 threads
    const int threads = threads_of(p.d, ni);
    if (ni == 1) return launch_norm<T, 1, 1024>(p, vec, threads, s);
    if (ni == 2) return launch_norm<T, 2, 1024>(p, vec, threads, s);
    if constexpr (sizeof(T) == 2)                        // floats have 4 groups from d = 16385 on
        if (threads <= 256) return launch_norm<T, 4, 256>(p, vec, threads, s);
    return launch_norm<T, 4, 1024>(p, vec, threads, s);
}

template <typename T>
bool vec_ok(const void *p, size_t ld) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && ld * sizeof(T) % 16 == 0);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const ds4c_rmsnorm_args &a, cudaStream_t s) {
    NormParams p{};
    p.n = (int)a.n;
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
    const bool gain_ok = ((uintptr_t)a.gain & 15) == 0;
    if (a.dtype == DS4C_F32) {
        using T = float;
        const bool vec = a.d % 8 == 0 && vec_ok<T>(a.x, a.x_ld) && vec_ok<T>(a.residual, a.residual_ld) &&
                         vec_ok<T>(a.residual_out, a.residual_out_ld) && vec_ok<T>(a.y_out, a.y_ld) && gain_ok;
        return launch_norm_t<T>(p, vec, s);
    }
    using T = __nv_bfloat16;
    const bool vec = a.d % 8 == 0 && vec_ok<T>(a.x, a.x_ld) && vec_ok<T>(a.residual, a.residual_ld) &&
                     vec_ok<T>(a.residual_out, a.residual_out_ld) && vec_ok<T>(a.y_out, a.y_ld) && gain_ok;
    return launch_norm_t<T>(p, vec, s);
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
