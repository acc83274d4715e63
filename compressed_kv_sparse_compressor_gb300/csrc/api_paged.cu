// extern "C" entry points of the attention over a paged cache (include/ds4c.h): argument validation on
// the host before any launch.
#include "ds4c_internal.cuh"

using namespace ds4c;

namespace {

constexpr uint32_t kMaxSeq = 4096, kMaxTokens = 1u << 20, kMaxHeads = 128;
constexpr size_t kMaxStride = (size_t)1 << 39;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool known_sizes(uint32_t n_seq, uint32_t n_tok, uint32_t n_heads, uint32_t d) {
    return n_seq <= kMaxSeq && n_tok <= kMaxTokens && n_heads >= 1 && n_heads <= kMaxHeads &&
           (d == 64 || d == 128 || d == 256 || d == 512);
}

ds4c_status check_pool(const ds4c_page_pool &p) {
    if (p.page_rows < 16 || p.page_rows > 1024 || (p.page_rows & (p.page_rows - 1)) != 0) return DS4C_ERR_SHAPE;
    if (p.n_pages == 0 || (uint64_t)p.n_pages * p.page_rows > 0x7fffffffull) return DS4C_ERR_SHAPE;
    if (p.max_pages > (1u << 27) || p.pages_ld < p.max_pages || p.pages_ld > kMaxStride) return DS4C_ERR_SHAPE;
    if (!p.rows || (!p.pages && p.max_pages > 0)) return DS4C_ERR_NULL;
    return aligned(p.rows, 16) && aligned(p.pages, 4) ? DS4C_OK : DS4C_ERR_SHAPE;
}

// Strides of [n][h] rows of d: multiples of 16 bytes, below the limit.
bool strides_ok(const ds4c_paged_attn_args &a, size_t token, size_t head) {
    return (a.n_tok <= 1 || (token % 8 == 0 && token > 0 && token < kMaxStride)) &&
           (a.n_heads <= 1 || (head % 8 == 0 && head > 0 && head < kMaxStride));
}
bool apart(size_t n_outer, size_t so, size_t n_inner, size_t si, size_t d) {
    return (n_inner <= 1 || si >= d) && (n_outer <= 1 || so >= (n_inner - 1) * si + d);
}

}  // namespace

extern "C" {

size_t ds4c_paged_attn_workspace_bytes(uint32_t n_seq, uint32_t n_tok, uint32_t n_heads, uint32_t head_dim) {
    return known_sizes(n_seq, n_tok, n_heads, head_dim) ? paged_attn_ws_bytes(n_seq, n_tok, n_heads, head_dim) : 0;
}

ds4c_status ds4c_paged_attn(const ds4c_paged_attn_args *args, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (!args) return DS4C_ERR_NULL;
    const ds4c_paged_attn_args &a = *args;
    if (!known_sizes(a.n_seq, a.n_tok, a.n_heads, a.head_dim)) return DS4C_ERR_SHAPE;
    if (!(a.scale > 0.f) || !(a.scale <= 1e4f) || a.window > 0x7fffffffu || a.ratio > 0x7fffffffu) return DS4C_ERR_SHAPE;
    if (a.n_seq == 0 || a.n_tok == 0) return DS4C_OK;
    if (!a.q || !a.out || !a.start || !a.length) return DS4C_ERR_NULL;
    if (a.q == a.out) return DS4C_ERR_SHAPE;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.start, 4) || !aligned(a.length, 4)) return DS4C_ERR_SHAPE;
    if (!strides_ok(a, a.q_token, a.q_head) || !strides_ok(a, a.out_token, a.out_head)) return DS4C_ERR_SHAPE;
    if (!apart(a.n_tok, a.out_token, a.n_heads, a.out_head, a.head_dim) &&
        !apart(a.n_heads, a.out_head, a.n_tok, a.out_token, a.head_dim))
        return DS4C_ERR_SHAPE;
    ds4c_status s = check_pool(a.raw);
    if (s == DS4C_OK && a.ratio) s = check_pool(a.comp);
    if (s != DS4C_OK) return s;
    if (!ws || !aligned(ws, 256) || ws_bytes < paged_attn_ws_bytes(a.n_seq, a.n_tok, a.n_heads, a.head_dim)) return DS4C_ERR_WORKSPACE;
    return cuda_status(launch_paged_attn(a, ws, stream));
}

}  // extern "C"
