// Attention of new tokens over a paged cache: a warp per token and head, one row after the other, online
// softmax.
#include <cuda_bf16.h>

#include "ds4c_internal.cuh"

namespace ds4c {

__device__ unsigned int g_paged_err;

namespace {

struct Pool {
    const __nv_bfloat16 *rows;
    const int32_t *pages;
    int64_t ld;
    int n_pages, page_rows, max_pages;
};
struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    int64_t q_token, q_head, out_token, out_head;
    const int32_t *start, *length;
    Pool raw, comp;
    int n_seq, n_tok, n_heads, window, ratio;
    float scale_log2;
};

template <int D>
__global__ void paged_attn_kernel(const Params p) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int E = D / 32;
    const int warp = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int token = warp / p.n_heads, h = warp % p.n_heads;
    if (token >= p.n_tok) return;
    for (int s = 0; s < p.n_seq; s++) {
        int b = p.start[s], e = p.start[s + 1];
        if (b < 0 || e < b || e > p.n_tok) {
            if (lane == 0) atomicOr(&g_paged_err, 2u);
            continue;
        }
        if (token < b || token >= e) continue;
        const int64_t t = (int64_t)p.length[s] - (e - b) + (token - b);
        float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
        for (int i = 0; i < E; i++) q[i] = __bfloat162float(p.q[token * p.q_token + h * p.q_head + lane + 32 * i]);
        for (int side = 0; side < 2; side++) {
            const Pool &pool = side ? p.comp : p.raw;
            int64_t lo = 0, hi = t + 1;
            if (side == 0 && p.window) lo = max((int64_t)0, t + 1 - p.window);
            if (side) hi = p.ratio && t >= 0 ? (t + 1) / p.ratio : 0;
            for (int64_t c = lo; c < hi; c++) {
                const int64_t k = c / pool.page_rows;
                const int page = k < pool.max_pages ? pool.pages[s * pool.ld + k] : -1;
                if (page < 0 || page >= pool.n_pages) {
                    if (lane == 0) atomicOr(&g_paged_err, 4u);
                    continue;
                }
                const __nv_bfloat16 *row = pool.rows + ((int64_t)page * pool.page_rows + c % pool.page_rows) * D;
                float x[E], dot = 0.f;
                for (int i = 0; i < E; i++) {
                    x[i] = __bfloat162float(row[lane + 32 * i]);
                    dot = fmaf(q[i], x[i], dot);
                }
                for (int w = 16; w; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
                dot *= p.scale_log2;
                const float mn = fmaxf(m, dot), f = exp2f(m - mn), pr = exp2f(dot - mn);
                for (int i = 0; i < E; i++) o[i] = fmaf(pr, x[i], o[i] * f);
                l = l * f + pr;
                m = mn;
            }
        }
        for (int i = 0; i < E; i++)
            p.out[token * p.out_token + h * p.out_head + lane + 32 * i] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
        return;
    }
}

Pool pool_of(const ds4c_page_pool &a) {
    return {static_cast<const __nv_bfloat16 *>(a.rows), a.pages, (int64_t)a.pages_ld, (int)a.n_pages, (int)a.page_rows, (int)a.max_pages};
}

}  // namespace

size_t paged_attn_ws_bytes(uint32_t, uint32_t, uint32_t, uint32_t) { return 256; }

cudaError_t launch_paged_attn(const ds4c_paged_attn_args &a, void *, cudaStream_t s) {
    Params p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.q_token = (int64_t)a.q_token; p.q_head = (int64_t)a.q_head;
    p.out_token = (int64_t)a.out_token; p.out_head = (int64_t)a.out_head;
    p.start = a.start; p.length = a.length;
    p.raw = pool_of(a.raw);
    if (a.ratio) p.comp = pool_of(a.comp);
    p.n_seq = (int)a.n_seq; p.n_tok = (int)a.n_tok; p.n_heads = (int)a.n_heads;
    p.window = (int)a.window; p.ratio = (int)a.ratio;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const dim3 grid((unsigned)(((uint64_t)a.n_tok * a.n_heads + 3) / 4));
    auto run = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(128), 0, s, p); };
    return a.head_dim == 64 ? run(paged_attn_kernel<64>) : a.head_dim == 128 ? run(paged_attn_kernel<128>)
         : a.head_dim == 256 ? run(paged_attn_kernel<256>) : run(paged_attn_kernel<512>);
}

unsigned int paged_attn_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof v) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_paged_err, &z, sizeof z);
    return v;
}

}  // namespace ds4c
