// extern "C" entry points of the 8-bit projections (include/ds4c.h): argument
// validation on the host before any launch.
#include "ds4c_internal.cuh"

using namespace ds4c;

namespace {

constexpr uint32_t kMaxRows = 1u << 24, kMaxSide = 1u << 18;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t elem_bytes(uint32_t dtype) { return dtype == DS4C_F32 ? 4 : 2; }
bool known(uint32_t dtype) { return dtype == DS4C_F32 || dtype == DS4C_BF16; }

// A matrix operand: optional, elements aligned, rows of d elements that do not overlap.
ds4c_status check_rows(const void *p, size_t ld, uint32_t d, uint32_t dtype) {
    if (!p) return DS4C_OK;
    return aligned(p, elem_bytes(dtype)) && ld >= d ? DS4C_OK : DS4C_ERR_SHAPE;
}

}  // namespace

extern "C" {

size_t ds4c_quant_row_bytes(uint32_t k) { return quant_row_bytes(k); }
size_t ds4c_quant_scale_bytes(uint32_t k) { return quant_scale_bytes(k); }

ds4c_status ds4c_rmsnorm_quant(const ds4c_rmsnorm_args *args, cudaStream_t stream) {
    if (!args) return DS4C_ERR_NULL;
    const ds4c_rmsnorm_args &a = *args;
    if (a.d == 0 || a.d > kMaxNormDim || !known(a.dtype) || a.n > kMaxRows) return DS4C_ERR_SHAPE;
    if (!(a.eps >= 1e-12f) || !(a.eps <= 1.f)) return DS4C_ERR_SHAPE;
    if (a.n == 0) return DS4C_OK;
    if (!a.q != !a.scale) return DS4C_ERR_NULL;
    if (!a.x || (!a.residual_out && !a.q && !a.y_out)) return DS4C_ERR_NULL;
    ds4c_status s;
    if ((s = check_rows(a.x, a.x_ld, a.d, a.dtype)) != DS4C_OK) return s;
    if ((s = check_rows(a.residual, a.residual_ld, a.d, a.dtype)) != DS4C_OK) return s;
    if ((s = check_rows(a.residual_out, a.residual_out_ld, a.d, a.dtype)) != DS4C_OK) return s;
    if ((s = check_rows(a.y_out, a.y_ld, a.d, a.dtype)) != DS4C_OK) return s;
    if (!aligned(a.gain, 4) || !aligned(a.q, 16) || !aligned(a.scale, 4)) return DS4C_ERR_SHAPE;
    // in place over x or the residual: the same rows, not shifted ones
    if (a.residual_out && a.residual_out == a.x && a.residual_out_ld != a.x_ld) return DS4C_ERR_SHAPE;
    if (a.residual_out && a.residual_out == a.residual && a.residual_out_ld != a.residual_ld) return DS4C_ERR_SHAPE;
    return cuda_status(launch_rmsnorm_quant(a, stream));
}

ds4c_status ds4c_quant_weight(uint32_t n, uint32_t k, uint32_t dtype, const void *w, size_t w_ld, uint8_t *q,
                              uint8_t *scale, cudaStream_t stream) {
    if (!w || !q || !scale) return DS4C_ERR_NULL;
    if (n == 0 || n > kMaxSide || k == 0 || k > kMaxSide || !known(dtype)) return DS4C_ERR_SHAPE;
    const ds4c_status s = check_rows(w, w_ld, k, dtype);
    if (s != DS4C_OK) return s;
    if (!aligned(q, 16) || !aligned(scale, 4)) return DS4C_ERR_SHAPE;
    return cuda_status(launch_quant_weight(n, k, dtype, w, w_ld, q, scale, stream));
}

ds4c_status ds4c_quant_matmul(uint32_t m, uint32_t k, const uint8_t *a, const uint8_t *a_scale,
                              const ds4c_quant_matrix *w, uint32_t n_w, uint32_t out_dtype, cudaStream_t stream) {
    if (!w) return DS4C_ERR_NULL;
    if (n_w == 0 || n_w > 4) return DS4C_ERR_UNSUPPORTED;
    if (m > kMaxRows || k == 0 || k > kMaxSide || !known(out_dtype)) return DS4C_ERR_SHAPE;
    if (m == 0) return DS4C_OK;
    if (!a || !a_scale) return DS4C_ERR_NULL;
    if (!aligned(a, 16) || !aligned(a_scale, 4)) return DS4C_ERR_SHAPE;
    QuantMatmulArgs q{};
    q.a = a;
    q.a_scale = a_scale;
    q.m = (int)m;
    q.k = (int)k;
    q.out_dtype = (int)out_dtype;
    q.n_w = (int)n_w;
    for (uint32_t g = 0; g < n_w; g++) {
        if (!w[g].q || !w[g].scale || !w[g].out) return DS4C_ERR_NULL;
        if (w[g].n == 0 || w[g].n > kMaxSide) return DS4C_ERR_SHAPE;
        if (!aligned(w[g].q, 16) || !aligned(w[g].scale, 4)) return DS4C_ERR_SHAPE;
        const ds4c_status s = check_rows(w[g].out, w[g].out_ld, w[g].n, out_dtype);
        if (s != DS4C_OK) return s;
        q.w[g] = w[g];
    }
    return cuda_status(launch_quant_matmul(q, stream));
}

}  // extern "C"
