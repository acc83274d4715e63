// Product of quantised rows with quantised weights on the 5th-generation tensor cores:
//   out_g[i][j] = sum_b 2^(ea[i][b] + ew_g[j / 128][b]) sum_{k in block b} a[i][k] w_g[j][k]
// for 1 to 4 weight matrices over the same rows, E4M3 codes, float accumulation.
//
// The scales are powers of two, so the tensor cores' block-scaled form (kind::mxf8f6f4,
// one E8M0 scale per operand row and 32 values of K) applies them in the product: a block
// of 128 values is four MMAs that name the same scale byte.  The weights are the MMA's
// M = 128 side and lie on the TMEM lanes, the rows are its N side: N follows the number
// of rows (16 for a single token), and a warp's 32 lanes hold 32 neighbouring outputs of
// one row, so the accumulator goes to global memory in whole lines straight from the
// registers.
//
//   - K in stages of 128 bytes (one scale block): the weights' [128][128] and the rows'
//     [BT][128] bytes by TMA in the 128-byte swizzle, a ring of mbarriers.  Rows and
//     columns past the ends, and K past the last value, are filled with zeros.
//   - Scales: the four scale bytes of 4 blocks of a row are read as a word, several groups of
//     4 blocks ahead, and lie in TMEM with row r's in lane r % 32 (of each lane quarter) and
//     column r / 32; the instruction descriptor picks the block's byte.  The split kernel
//     copies the words to shared memory (cp.async) and from there to TMEM (tcgen05.cp); the
//     pair kernel writes TMEM from registers, see there.
//   - A cluster of `split` CTAs shares an output tile, each with a range of K; the
//     partial tiles meet through distributed shared memory and are added in rank order.
//   - The tensor core's float accumulation cuts low bits off (the error grows with K: 4e-7 of
//     the result's norm at K = 4096), so an accumulator takes at most CHUNK blocks of K; two
//     take turns, and the epilogue adds the chunks in registers.
//   - Every mbarrier wait is bounded; a wait that gives up raises the library's device
//     error word and the CTA winds down, freeing its tensor memory.
//
// What bounds it, on inputs that are not in L2: few rows, the weights' bytes and the chain
// launch - loads - MMAs - meeting (one row through 2560 x 4096 weights 4.9 us for 1.5 us of
// bytes, through 8192 x 8192 14.0 us, 4.8 TB/s); many rows, the ring of loads (about 3000
// cycles from a stage's release to its next data) and then the tensor pipe and the power
// limit (8192 x 8192 x 8192 305 us, 3.6 PFLOP/s; 352-359 us, 3.1 PFLOP/s, at 1.35 GHz when run
// for seconds).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <atomic>

#include "ds4c_internal.cuh"

namespace ds4c {

__device__ unsigned int g_qmm_err;
__device__ unsigned long long g_qmm_wait_ns = kWaitNsDefault;

namespace {

constexpr int BW = 128, BK = 128;              // weight rows and K bytes of a stage
constexpr int THREADS = 256;
constexpr int SF_SLOTS = 5;                    // groups of 4 stages whose scales shared memory and TMEM hold
constexpr int SF_AHEAD = 3;                    // groups whose copies are in flight (below SF_SLOTS)
constexpr int SF_BYTES = 512;                  // scales of 128 rows, 4 stages
constexpr int CHUNK = 32;                      // blocks of K that one accumulator takes

template <int BT>
struct Shape {
    static constexpr int W_BYTES = BW * BK, T_BYTES = BT * BK, STAGE_BYTES = W_BYTES + T_BYTES;
    // BT <= 64: two CTAs to an SM, so that one's loads cover the other's start and end
    static constexpr int PER_SM = BT <= 64 ? 2 : 1;
    static constexpr int STAGES = BT <= 32 ? 5 : BT <= 64 ? 4 : 6;
    static constexpr int SFT = (BT + 127) / 128;               // 128-row units of the rows' scales
    static constexpr int SF_SLOT_BYTES = SF_BYTES * (1 + SFT);
    static constexpr int SF_COLS = 4 * (1 + SFT);
    static constexpr int COLS = 2 * BT + SF_SLOTS * SF_COLS;
    static constexpr int TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr int N_BARS = 2 * STAGES + 2 * SF_SLOTS + 5;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SF_SLOTS * SF_SLOT_BYTES + 8 * N_BARS + 16 + 1024;
    // instruction descriptor: A = B = E4M3, both K-major, E8M0 scales, M = 128, N = BT; the
    // scale byte's index goes to bits 4 (B) and 29 (A)
    static constexpr uint32_t IDESC = ((uint32_t)(BT >> 3) << 17) | (1u << 23) | ((uint32_t)(BW >> 7) << 27);
    static_assert(BT % 16 == 0 && BT <= 256, "MMA N");
    // the last stages hold the partial sums that a CTA receives,
    // from 8 CTAs, at least 4 rows each
    static constexpr int PART_STAGES = ((BT < 32 ? 32 : BT) * BW * 4 + STAGE_BYTES - 1) / STAGE_BYTES;
    static_assert(PART_STAGES < STAGES, "the partial sums reuse stages");
    static_assert(PER_SM * TMEM_COLS <= 512, "TMEM of the CTAs of an SM");
    static_assert(PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "CTAs to an SM");
};

struct Params {
    const uint8_t *a_scale;
    int m, kb;                   // rows, scale blocks of K
    int k_tail;                  // MMAs (32 values each) of the last block
    int scale_ld;
    int m_tiles, n_w, bf16_out;
    int tile_start[5];           // prefix sums of output tiles per weight matrix
    int n[4];
    const uint8_t *w_scale[4];
    void *out[4];
    int64_t out_ld[4];
};
struct Maps { CUtensorMap a, w[4]; };

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Counts `bytes` as if a copy had brought them.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity);
// Bounded wait of a whole warp for the completion of the phase with the given parity (CLUSTER: of arrivals
// from both CTAs of a pair, whose writes it acquires).  (A vote on the first look and then each lane for itself:
// 1024 x 4096 x 4096 17.8 us for 17.2, 32 rows 5.85 for 5.7.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return warp_bounded_wait<256>([=] { return CLUSTER ? mbar_try_cluster(bar, parity) : mbar_try(bar, parity); }, abort,
                                  g_qmm_wait_ns, &g_qmm_err);
}
// Bounded wait that ignores the abort flag: drains copies or MMAs still in
// flight after a give-up, before the CTA frees its TMEM and exits.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (mbar_try(bar, parity)) return;
        if ((i & 255u) == 255u) {
            const uint64_t now = globaltimer();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kDrainNs) return;
        }
    }
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Pair forms: an mbarrier of CTA `rank` of the cluster, arrivals and waits that order memory
// across the pair, loads that complete on the leader's barrier, commits to both CTAs.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Without memory ordering: for a barrier that guards TMEM only, which tcgen05.fence orders.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// Brings a box to L2.  Made before the wait for the previous kernel: L2 holds one copy of memory, so a
// box that kernel still writes is read as written later.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x),
                 "r"(y)
                 : "memory");
}
// Shared-memory matrix descriptors: K-major operand in the 128-byte swizzle TMA writes
// (8-row atoms of 1024 bytes), and the unswizzled scale words (8-row cores of 128 bytes).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ void cluster_st(uint32_t addr, uint32_t rank, uint32_t v) {
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(mapa(addr, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_st4(uint32_t addr, uint32_t rank, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mapa(addr, rank)), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

// Copies the scale words of group q (4 stages) of 128 rows, row r of them at src + r * ld, into their
// slot; rows from `rows` on get zero bytes (their codes are zeros too).  One warp.
__device__ __forceinline__ void copy_words(uint32_t dst, const uint8_t *src, int ld, int rows, int q, int lane) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int r = j * 32 + lane;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + lane * 16 + j * 4),
                     "l"(r < rows ? src + (size_t)r * ld + 4 * q : src), "r"(r < rows ? 4 : 0)
                     : "memory");
    }
}
// The same with one word for all rows.
__device__ __forceinline__ void copy_word(uint32_t dst, const uint8_t *src, int q, int lane) {
#pragma unroll
    for (int j = 0; j < 4; j++)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + lane * 16 + j * 4), "l"(src + 4 * q) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` groups of this thread's copies are in flight, and shows the others to
// the asynchronous proxy.
template <int left>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void store_out(void *out, int64_t i, float v, int bf16) {
    if (bf16) static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(out)[i] = v;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
// A thread's column of the output: v's first `rows` values to rows of pitch ld.  Groups of 16 without a
// check between them where the rows allow: with a check and a 64-bit product for each value this
// took three quarters of an 8192 x 8192 x 512 product's time.
template <typename T, int N>
__device__ __forceinline__ void store_column(T *out, int64_t ld, const float (&v)[N][16], int rows) {
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (16 * i + 16 <= rows) {
#pragma unroll
            for (int j = 0; j < 16; j++, out += ld) put(out, v[i][j]);
        } else if (16 * i < rows) {
#pragma unroll
            for (int j = 0; j < 16; j++, out += ld)
                if (16 * i + j < rows) put(out, v[i][j]);
        }
    }
}

template <int BT>
__global__ void __launch_bounds__(THREADS, 1) qmm_split_kernel(const __grid_constant__ Maps maps, const Params p, int split) {
    using S = Shape<BT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sf = smem + S::STAGES * S::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(sf + SF_SLOTS * S::SF_SLOT_BYTES);
    uint64_t *empty = full + S::STAGES, *sf_full = empty + S::STAGES, *sf_empty = sf_full + SF_SLOTS;
    uint64_t *acc_full = sf_empty + SF_SLOTS, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    const int rank = (int)blockIdx.x % split, tile = (int)blockIdx.x / split;
    int g = 0;
    while (g + 1 < p.n_w && tile >= p.tile_start[g + 1]) g++;
    const int nt = (tile - p.tile_start[g]) / p.m_tiles, m0 = (tile - p.tile_start[g]) % p.m_tiles * BT;
    const int n0 = nt * BW;
    // the K ranges of the ranks differ by at most one block
    const int kb0 = (int)((int64_t)p.kb * rank / split), kb1 = (int)((int64_t)p.kb * (rank + 1) / split);
    // Meeting: each CTA adds the groups of 4 rows whose number is its rank modulo split (a power of two), to
    // which the others write their partial sums, into the last stages: free from the start if no CTA's K
    // comes that far (`unused`), else once all MMAs of the cluster are done.  The cluster barrier's first
    // phase says that, the second that the sums have arrived.  (The sums of 32 rows through 2560 x 4096 weights
    // read from the other CTAs instead, a round trip more: 6.65 us for 5.9; sent value by value, 128 rows:
    // 11 us for 9.4.)
    const int log_split = 31 - __clz(split), own = max(1, BT / 4 >> log_split);
    const bool unused = (p.kb + split - 1) >> log_split <= S::STAGES - S::PART_STAGES;
    float4 *part = reinterpret_cast<float4 *>(smem + (S::STAGES - S::PART_STAGES) * S::STAGE_BYTES);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; s++) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < SF_SLOTS; s++) {
            mbar_init(smem_u32(&sf_full[s]), 32);
            mbar_init(smem_u32(&sf_empty[s]), 1);
        }
        for (int a = 0; a < 2; a++) {
            mbar_init(smem_u32(&acc_full[a]), 1);
            mbar_init(smem_u32(&acc_empty[a]), 4);
        }
        mbar_init(smem_u32(drain), 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(S::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    if (BT <= 32 && warp == 3 && (int)gridDim.x / split * p.kb >= 256 && elect()) {
        // the weights of the first stages, while the previous kernel ends, beside which these small CTAs can
        // start.  For weights of 4 MB on (32 rows, K = 1024: 8192 columns 5.4 -> 5.0 us, but 2560 3.65 -> 3.9;
        // 2560 x 4096 6.1 -> 5.9) and tiles of up to 32 rows (64 rows: 2560 x 4096 8.0 -> 7.4, but 4096 x 4096
        // 7.9 -> 8.6)
        for (int kb = kb0; kb < min(kb1, kb0 + S::STAGES); kb++) tma_prefetch_2d(&maps.w[g], kb * BK, n0);
    }
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    if (split > 1 && unused) cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();

    // warps 0 and 1 run converged and one elected lane issues, so that what the copies and MMAs take lies
    // in uniform registers
    uint32_t filled = 0;                             // warp 0's: stages it filled
    if (warp == 0) {
        uint32_t it = 0, s = 0, par = 1;
        const uint32_t base = smem_u32(smem);
        const CUtensorMap *mw = &maps.w[g];
        for (int kb = kb0; kb < kb1; kb++, it++) {
            if (!warp_wait(smem_u32(&empty[s]), par, abort)) break;
            const uint32_t bar = smem_u32(&full[s]), dst = base + s * S::STAGE_BYTES;
            if (elect()) {
                mbar_expect_tx(bar, S::STAGE_BYTES);
                tma_load_2d(dst, mw, kb * BK, n0, bar);
                tma_load_2d(dst + S::W_BYTES, &maps.a, kb * BK, m0, bar);
            }
            __syncwarp();
            if (++s == S::STAGES) s = 0, par ^= 1;
        }
        filled = it;
        __syncwarp();
    } else if (warp == 1) {
        uint32_t s = 0, s_par = 0, sl = 0, accumulate = 0;
        const uint32_t sf_tmem = tmem + 2 * BT;
        const uint64_t w_desc = sw128_desc(smem_u32(smem)), sf_desc = scale_desc(smem_u32(sf));
        for (int kb = kb0; kb < kb1; kb++) {
            const uint32_t slot = sl % SF_SLOTS, c = (uint32_t)(kb - kb0) / CHUNK, acc = c & 1, d = tmem + acc * BT;
            const uint32_t sfa = sf_tmem + slot * S::SF_COLS, sfb = sfa + 4;
            if ((kb - kb0) % CHUNK == 0) {
                if (!warp_wait(smem_u32(&acc_empty[acc]), ((c >> 1) & 1) ^ 1, abort)) break;
                fence_after();
                accumulate = 0;
            }
            if (kb == kb0 || kb % 4 == 0) {
                if (!warp_wait(smem_u32(&sf_full[slot]), (sl / SF_SLOTS) & 1, abort)) break;
                fence_after();
                const uint64_t src = sf_desc + (uint64_t)(slot * (S::SF_SLOT_BYTES >> 4));
                if (elect()) {
#pragma unroll
                    for (int i = 0; i < 1 + S::SFT; i++) copy_scales(sfa + 4 * i, src + (uint64_t)(i * (SF_BYTES >> 4)));
                }
                __syncwarp();
            }
            if (!warp_wait(smem_u32(&full[s]), s_par, abort)) break;
            fence_after();
            const uint64_t wd = w_desc + (uint64_t)(s * (S::STAGE_BYTES >> 4)), td = wd + (S::W_BYTES >> 4);
            const uint32_t id = (uint32_t)kb % 4, idesc = S::IDESC | id << 4 | id << 29;
            const bool group_end = kb % 4 == 3;
            if (elect()) {
                if (kb < p.kb - 1 || p.k_tail == BK / 32) {
#pragma unroll
                    for (int k = 0; k < BK / 32; k++)
                        mma_scaled(d, wd + 2 * k, td + 2 * k, idesc, sfa, sfb, k > 0 ? 1u : accumulate);
                } else {
                    for (int k = 0; k < p.k_tail; k++)
                        mma_scaled(d, wd + 2 * k, td + 2 * k, idesc, sfa, sfb, k > 0 ? 1u : accumulate);
                }
                mma_commit(smem_u32(&empty[s]));
                if (group_end) mma_commit(smem_u32(&sf_empty[slot]));
                if ((kb - kb0) % CHUNK == CHUNK - 1 || kb == kb1 - 1) mma_commit(smem_u32(&acc_full[acc]));
            }
            __syncwarp();
            accumulate = 1;
            sl += group_end ? 1 : 0;
            if (++s == S::STAGES) s = 0, s_par ^= 1;
        }
        // the drain: every MMA issued so far completes (bounded wait, given up or not) before the
        // TMEM is freed
        if (elect()) mma_commit(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0);
        __syncwarp();
    } else if (warp == 2) {
        // scales of groups of 4 stages (absolute positions, so a group is one word per row)
        const uint8_t *ws = p.w_scale[g] + (size_t)nt * p.scale_ld, *ts = p.a_scale + (size_t)m0 * p.scale_ld;
        uint32_t issued = 0, done = 0;
        for (int q = kb0 / 4; q < (kb1 + 3) / 4; q++, issued++) {
            const int slot = issued % SF_SLOTS;
            if (!warp_wait(smem_u32(&sf_empty[slot]), ((issued / SF_SLOTS) & 1) ^ 1, abort)) break;
            const uint32_t dst = smem_u32(sf + slot * S::SF_SLOT_BYTES);
            copy_word(dst, ws, q, lane);
#pragma unroll
            for (int i = 0; i < S::SFT; i++)
                copy_words(dst + (1 + i) * SF_BYTES, ts + (size_t)i * 128 * p.scale_ld, p.scale_ld, min(BT, p.m - m0) - i * 128, q,
                           lane);
            copies_commit();
            if (issued - done == SF_AHEAD) {
                copies_wait<SF_AHEAD>();
                mbar_arrive(smem_u32(&sf_full[done++ % SF_SLOTS]));
            }
        }
        copies_wait<0>();
        for (; done < issued; done++) mbar_arrive(smem_u32(&sf_full[done % SF_SLOTS]));
        __syncwarp();
    } else if (warp >= 4) {
        // epilogue: TMEM lane quarter warp % 4, lane = weight row, column = row of the product
        const int quarter = warp & 3, n = n0 + quarter * 32 + lane;
        const int rows = min(BT, p.m - m0);
        float v[BT / 16][16];
        bool ok = true;
        const int chunks = (kb1 - kb0 + CHUNK - 1) / CHUNK;
        for (int c = 0; c < chunks; c++) {
            const uint32_t acc = c & 1, src = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BT;
            ok = warp_wait(smem_u32(&acc_full[acc]), (c >> 1) & 1, abort);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int i = 0; i < BT / 16; i++)
                if (16 * i < rows) {
                    if (c == 0) {
                        tmem_ld16(src + 16 * i, v[i]);
                    } else {
                        float u[16];
                        tmem_ld16(src + 16 * i, u);
#pragma unroll
                        for (int j = 0; j < 16; j++) v[i][j] += u[j];
                    }
                }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&acc_empty[acc]));
            __syncwarp();
        }
        if (split > 1) {
            __syncwarp();
            if (!unused) cluster_arrive();
            cluster_wait();
            const uint32_t dst = smem_u32(part + rank * own * BW + quarter * 32 + lane);
#pragma unroll
            for (int q = 0; q < BT / 4; q++)
                if (ok && 4 * q < rows)
                    cluster_st4(dst + (q >> log_split) * (BW * 16), q & (split - 1), v[q / 4][q % 4 * 4], v[q / 4][q % 4 * 4 + 1],
                                v[q / 4][q % 4 * 4 + 2], v[q / 4][q % 4 * 4 + 3]);
        } else if (ok && n < p.n[g]) {
            const int64_t ld = p.out_ld[g], o = (int64_t)m0 * ld + n;
            if (p.bf16_out) store_column(static_cast<__nv_bfloat16 *>(p.out[g]) + o, ld, v, rows);
            else store_column(static_cast<float *>(p.out[g]) + o, ld, v, rows);
        }
    }
    if (split > 1) {
        // partial sums [source][own group][128 columns][4 rows], added in rank order
        __syncwarp();
        if (warp < 4) {
            if (!unused) cluster_arrive();
            cluster_wait();
        }
        cluster_sync();
        const int rows = min(BT, p.m - m0), total = (((rows + 3) / 4 - rank + split - 1) >> log_split) * BW;
        for (int e = threadIdx.x; e < total; e += THREADS) {
            float4 u[8];                                 // every load in flight before the first addition
#pragma unroll
            for (int r = 0; r < 8; r++)
                if (r < split) u[r] = part[r * own * BW + e];
            float4 v = u[0];
#pragma unroll
            for (int r = 1; r < 8; r++)
                if (r < split) v.x += u[r].x, v.y += u[r].y, v.z += u[r].z, v.w += u[r].w;
            const int n = n0 + e % BW, row = ((e / BW << log_split) + rank) * 4;
            if (n >= p.n[g]) continue;
            int64_t o = (int64_t)(m0 + row) * p.out_ld[g] + n;
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; j++, o += p.out_ld[g])
                if (row + j < rows) store_out(p.out[g], o, f[j], p.bf16_out);
        }
    }
    __syncthreads();
    // after a give-up of any warp the MMAs may not have waited for every load: the last STAGES land before the CTA exits
    if (warp == 0 && *abort)
        for (uint32_t u = filled > (uint32_t)S::STAGES ? filled - S::STAGES : 0; u < filled; u++)
            mbar_drain(smem_u32(&full[u % S::STAGES]), (u / S::STAGES) & 1);
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------------------------------
// Large products: a persistent kernel of CTA pairs.  cta_group::2 MMAs of 256 weight rows x
// bt rows: each CTA holds 128 weight rows and half of the rows in shared memory, so a stage
// costs (128 + bt / 2) * 128 bytes of loads per SM where one CTA alone would need
// (128 + bt) * 128.  bt (a multiple of 32, at most 224) is chosen by the host so that the
// tiles fill whole rounds over the pairs; two accumulators of bt columns and five slots of
// scales fit the 512 TMEM columns, so a tile's epilogue runs beside the next tile's MMAs.
//
// Warps: 0 loads (in both CTAs, completing on the leader's barriers), 1 MMAs (leader only),
// 4-11 epilogue (TMEM lane quarter w % 4, half of the columns each), 12-15 scales (in both
// CTAs, the words of all bt rows and of the CTA's own weight rows to lane quarter w % 4).
// ---------------------------------------------------------------------------------------
constexpr int PAIR_THREADS = 512, MAX_BT = 224;
// registers per thread of the epilogue's two warpgroups and of the other two (setmaxnreg), out of 128 at launch
constexpr int REG_EPILOGUE = 168, REG_OTHER = 80;
constexpr uint32_t NOT_ISSUED = ~0u;
constexpr int PAIR_STAGES = 8, PAIR_RING = 216 * 1024;       // most stages, bytes of the ring
struct Pair {
    static constexpr int W_BYTES = BW * BK;
    static constexpr int SF_COLS = 12, WORDS = MAX_BT / 32;      // TMEM columns of a slot, row words of a lane
    static constexpr int N_BARS = 2 * PAIR_STAGES + 2 * SF_SLOTS + 5;
    static constexpr int SMEM_BYTES = PAIR_RING + 8 * N_BARS + 16 + 1024;      // 16: TMEM address, abort, issued[2]
    static constexpr uint32_t IDESC = (1u << 23) | ((uint32_t)(2 * BW >> 7) << 27);       // M = 256, N added
    static constexpr int HALF_CHUNKS = MAX_BT / 2 / 16;
    static_assert(2 * MAX_BT + SF_SLOTS * SF_COLS <= 512, "TMEM columns");
    static_assert(2 * REG_EPILOGUE + 2 * REG_OTHER <= 4 * 128, "registers of the four warpgroups");
    static_assert(7 * (W_BYTES + MAX_BT / 2 * BK) <= PAIR_RING && SMEM_BYTES <= 232448, "seven stages at the widest tile");
};

// Output tile -> weight matrix, row tile and weight tile: within a matrix, 16 weight tiles go
// with each row tile before the next row tile, so that the tiles in flight share their operands in L2.
__device__ __forceinline__ void pair_coords(const Params &p, int tile, int &g, int &mt, int &nt) {
    g = 0;
    while (g + 1 < p.n_w && tile >= p.tile_start[g + 1]) g++;
    const int local = tile - p.tile_start[g], n_tiles = (p.n[g] + 2 * BW - 1) / (2 * BW);
    const int band = local / (16 * p.m_tiles), wide = min(16, n_tiles - 16 * band);
    const int in = local - band * 16 * p.m_tiles;
    mt = in / wide;
    nt = 16 * band + in % wide;
}

__device__ __forceinline__ uint32_t load_word(const uint8_t *p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// A warp's scale words of group q (4 blocks of K): lane l holds row 32 j + l's word in t[j], the weight
// tile's in w.  Rows from `rows` on get zeros (their codes are zeros too).
struct ScaleWords { uint32_t w, t[Pair::WORDS]; };
__device__ __forceinline__ void load_scales(ScaleWords &s, const uint8_t *ws, const uint8_t *ts, int ld, int rows, int q,
                                            int lane) {
    s.w = load_word(ws + 4 * q);
#pragma unroll
    for (int j = 0; j < Pair::WORDS; j++)
        s.t[j] = 32 * j + lane < rows ? load_word(ts + (size_t)(32 * j + lane) * ld + 4 * q) : 0u;
}
// ... to this warp's lane quarter of a TMEM slot: four columns of the weights' word, eight of the rows'.
__device__ __forceinline__ void store_scales(uint32_t taddr, const ScaleWords &s) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(taddr), "r"(s.w) : "memory");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr + 4), "r"(s.t[0]),
                 "r"(s.t[1]), "r"(s.t[2]), "r"(s.t[3]), "r"(s.t[4]), "r"(s.t[5]), "r"(s.t[6]), "r"(0u)
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
static_assert(Pair::WORDS == 7, "columns of store_scales");

// The pair's loads land before it exits where the leader's MMAs gave up (else they have waited for every load).  Both
// CTAs' loads complete on the leader's barriers, so its MMA warp waits for both: issued[r] says how many stages CTA r
// filled, and a stage that only one filled gets the other's part of its count here.
__device__ __forceinline__ void pair_drain(uint32_t full, volatile uint32_t *issued, uint32_t stages, uint32_t block, int kb,
                                           bool joint) {
    // the loading warps' waits are bounded too, so that the counts come
    const uint64_t t0 = globaltimer();
    while ((issued[0] == NOT_ISSUED || issued[1] == NOT_ISSUED) && globaltimer() - t0 <= 2 * kDrainNs) {}
    __syncwarp();
    uint32_t n0 = __shfl_sync(0xffffffffu, issued[0], 0), n1 = __shfl_sync(0xffffffffu, issued[1], 0);
    if (n0 == NOT_ISSUED) n0 = n1;                   // only where the wait limit was set beyond this one's
    if (n1 == NOT_ISSUED) n1 = n0;
    if (n0 == NOT_ISSUED) return;
    const uint32_t n = max(n0, n1), per_tile = joint ? (kb + 1) / 2 : kb;
    for (uint32_t u = n > stages ? n - stages : 0; u < n; u++) {
        const uint32_t bar = full + 8 * (u % stages);
        // what one CTA brings: a stage of two blocks of K but at the end of an odd number of them
        const uint32_t bytes = joint && !(kb % 2 == 1 && u % per_tile == per_tile - 1) ? 2 * block : block;
        if (elect()) {
            if (u >= n0) mbar_expect_tx(bar, bytes);
            else if (u >= n1) mbar_complete_tx(bar, bytes);
        }
        __syncwarp();
        mbar_drain(bar, (u / stages) & 1);
        __syncwarp();
    }
}

template <bool joint>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
qmm_pair_kernel(const __grid_constant__ Maps maps, const Params p, int bt) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + PAIR_RING);
    uint64_t *empty = full + PAIR_STAGES, *sf_full = empty + PAIR_STAGES, *sf_empty = sf_full + SF_SLOTS;
    uint64_t *acc_full = sf_empty + SF_SLOTS, *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile uint32_t *issued = tmem_slot + 2;       // the leader's: stages that each CTA filled, once that is known
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int rank = (int)blockIdx.x & 1, pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
    const int total = p.tile_start[p.n_w], chunks = (p.kb + CHUNK - 1) / CHUNK;
    // The MMA warp takes two blocks of K at a time.  A stage is one block for wide tiles (!joint), whose
    // seven keep more loads in flight than three stages of two would; two blocks for narrow ones (up to 160
    // rows), whose MMAs (2 bt cycles a block) are shorter than a stage's handshakes (8192 x 8192 x 8192 on
    // zeros: 224 rows 251 us in stages of one block and 284 of two, 128 rows 347 and 327)
    const uint32_t block = Pair::W_BYTES + (uint32_t)bt / 2 * BK, stage = joint ? 2 * block : block;
    const uint32_t stages = min((uint32_t)PAIR_STAGES, PAIR_RING / stage);

    if (threadIdx.x == 0) {
        for (int s = 0; s < PAIR_STAGES; s++) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < SF_SLOTS; s++) {
            mbar_init(smem_u32(&sf_full[s]), 8);
            mbar_init(smem_u32(&sf_empty[s]), 1);
        }
        for (int a = 0; a < 2; a++) {
            mbar_init(smem_u32(&acc_full[a]), 1);
            mbar_init(smem_u32(&acc_empty[a]), 16);
        }
        mbar_init(smem_u32(drain), 1);
        *abort = 0;
        issued[0] = issued[1] = NOT_ISSUED;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        fence_before();
    }
    __syncthreads();
    cluster_sync();                                  // both CTAs' barriers exist before either uses them
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    // each warpgroup resizes its registers once, its four warps together; the host checked the launch's share
    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
    if (warp == 0) {
        bool ok = true;
        uint32_t it = 0, s = 0, par = 1;
        const uint32_t base = smem_u32(smem), full0 = mapa(smem_u32(full), 0);
        for (int tile = pair; tile < total && ok; tile += pairs) {
            int g, mt, nt;
            pair_coords(p, tile, g, mt, nt);
            const int wy = nt * 2 * BW + rank * BW, ty = mt * bt + rank * (bt / 2);
            const CUtensorMap *mw = &maps.w[g];
            for (int kb = 0; kb < p.kb; kb += joint ? 2 : 1, it++) {
                if (!warp_wait<true>(smem_u32(&empty[s]), par, abort)) { ok = false; break; }
                const uint32_t dst = base + s * stage, bar = full0 + 8 * s;
                const bool two = joint && kb + 1 < p.kb;
                if (elect()) {
                    if (rank == 0) mbar_expect_tx(smem_u32(&full[s]), (two ? 4 : 2) * block);
                    tma_load_2d_pair(dst, mw, kb * BK, wy, bar);
                    tma_load_2d_pair(dst + Pair::W_BYTES, &maps.a, kb * BK, ty, bar);
                    if (two) {
                        tma_load_2d_pair(dst + block, mw, kb * BK + BK, wy, bar);
                        tma_load_2d_pair(dst + block + Pair::W_BYTES, &maps.a, kb * BK + BK, ty, bar);
                    }
                }
                __syncwarp();
                if (++s == stages) s = 0, par ^= 1;
            }
        }
        if (elect()) cluster_st(smem_u32(tmem_slot + 2 + rank), 0, it);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            bool ok = true;
            uint32_t s = 0, s_par = 0, sl = 0, local = 0;
            const uint32_t sf_tmem = tmem + 2 * (uint32_t)bt;
            const uint32_t idesc0 = Pair::IDESC | (uint32_t)(bt >> 3) << 17;
            const uint64_t w_desc = sw128_desc(smem_u32(smem));
            for (int tile = pair; tile < total && ok; tile += pairs) {
                for (int c = 0; c < chunks && ok; c++, local++) {
                    const uint32_t acc = local & 1, d = tmem + acc * (uint32_t)bt;
                    if (!warp_wait<true>(smem_u32(&acc_empty[acc]), ((local >> 1) & 1) ^ 1, abort)) { ok = false; break; }
                    fence_after();
                    const int kb1 = min(p.kb, (c + 1) * CHUNK);
                    uint32_t accumulate = 0;
                    for (int kb = c * CHUNK; kb < kb1; kb += 2) {
                        const uint32_t slot = sl % SF_SLOTS;
                        const uint32_t sfa = sf_tmem + slot * Pair::SF_COLS, sfb = sfa + 4;
                        if (kb % 4 == 0) {
                            if (!warp_wait<true>(smem_u32(&sf_full[slot]), (sl / SF_SLOTS) & 1, abort)) { ok = false; break; }
                            fence_after();
                        }
                        const bool two = kb + 1 < p.kb;
                        // the second block's stage
                        const uint32_t s1 = joint ? s : s + 1 == stages ? 0 : s + 1, par1 = s + 1 == stages ? s_par ^ 1 : s_par;
                        if (!warp_wait<true>(smem_u32(&full[s]), s_par, abort)) { ok = false; break; }
                        if (!joint && two && !warp_wait<true>(smem_u32(&full[s1]), par1, abort)) { ok = false; break; }
                        fence_after();
                        const uint64_t wd = w_desc + (uint64_t)(s * (stage >> 4));
                        const uint64_t wd1 = joint ? wd + (block >> 4) : w_desc + (uint64_t)(s1 * (stage >> 4));
                        constexpr uint64_t T = Pair::W_BYTES >> 4;
                        const uint32_t id = (uint32_t)kb % 4, idesc = idesc0 | id << 4 | id << 29, idesc1 = idesc + (1u << 4 | 1u << 29);
                        const bool group_end = kb % 4 == 2 || kb + 2 >= p.kb;
                        if (elect()) {
                            if (kb + 2 < p.kb || (kb + 2 == p.kb && p.k_tail == BK / 32)) {
#pragma unroll
                                for (int k = 0; k < BK / 32; k++)
                                    mma_scaled_pair(d, wd + 2 * k, wd + T + 2 * k, idesc, sfa, sfb, k > 0 ? 1u : accumulate);
                                if (!joint) mma_commit_pair(smem_u32(&empty[s]));
#pragma unroll
                                for (int k = 0; k < BK / 32; k++)
                                    mma_scaled_pair(d, wd1 + 2 * k, wd1 + T + 2 * k, idesc1, sfa, sfb, 1u);
                            } else {                     // the last one or two blocks, the last one shorter
                                const int n0 = two ? BK / 32 : p.k_tail, n1 = two ? p.k_tail : 0;
                                for (int k = 0; k < n0; k++)
                                    mma_scaled_pair(d, wd + 2 * k, wd + T + 2 * k, idesc, sfa, sfb, k > 0 ? 1u : accumulate);
                                if (!joint) mma_commit_pair(smem_u32(&empty[s]));
                                for (int k = 0; k < n1; k++)
                                    mma_scaled_pair(d, wd1 + 2 * k, wd1 + T + 2 * k, idesc1, sfa, sfb, 1u);
                            }
                            if (two || joint) mma_commit_pair(smem_u32(&empty[s1]));
                            if (group_end) mma_commit_pair(smem_u32(&sf_empty[slot]));
                        }
                        __syncwarp();
                        accumulate = 1;
                        sl += group_end ? 1 : 0;
                        s += two && !joint ? 2 : 1;
                        if (s >= stages) s -= stages, s_par ^= 1;
                    }
                    if (ok && elect()) mma_commit_pair(smem_u32(&acc_full[acc]));
                    __syncwarp();
                }
            }
            // drain: every MMA issued so far completes (bounded wait, given up or not) before the
            // TMEM is freed
            if (elect()) mma_commit_pair(smem_u32(drain));
            __syncwarp();
            mbar_drain(smem_u32(drain), 0);
            __syncwarp();
            if (!ok) pair_drain(smem_u32(full), issued, stages, block, p.kb, joint);
        }
        __syncwarp();
    }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_EPILOGUE));
        const int quarter = warp & 3, half = (warp - 4) / 4, cols = bt / 2;
        uint32_t local = 0;
        bool ok = true;
        for (int tile = pair; tile < total && ok; tile += pairs) {
            int g, mt, nt;
            pair_coords(p, tile, g, mt, nt);
            float v[Pair::HALF_CHUNKS][16];
            for (int c = 0; c < chunks; c++, local++) {
                const uint32_t acc = local & 1;
                ok = warp_wait<true>(smem_u32(&acc_full[acc]), (local >> 1) & 1, abort);
                if (!ok) break;
                fence_after();
                const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + acc * (uint32_t)bt + (uint32_t)(half * cols);
#pragma unroll
                for (int i = 0; i < Pair::HALF_CHUNKS; i++) {
                    if (16 * i < cols) {
                        if (c == 0) {
                            tmem_ld16(src + 16 * i, v[i]);
                        } else {
                            float u[16];
                            tmem_ld16(src + 16 * i, u);
#pragma unroll
                            for (int j = 0; j < 16; j++) v[i][j] += u[j];
                        }
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(mapa(smem_u32(&acc_empty[acc]), 0));
                __syncwarp();
            }
            if (!ok) break;
            const int n = nt * 2 * BW + rank * BW + quarter * 32 + lane, m0 = mt * bt + half * cols;
            if (n < p.n[g]) {
                const int64_t ld = p.out_ld[g], o = (int64_t)m0 * ld + n;
                const int rows = min(cols, p.m - m0);
                if (p.bf16_out) store_column(static_cast<__nv_bfloat16 *>(p.out[g]) + o, ld, v, rows);
                else store_column(static_cast<float *>(p.out[g]) + o, ld, v, rows);
            }
            __syncwarp();                                // the next wait and loads are the whole warp's
        }
        __syncwarp();
    } else {
        // Scales: each of four warps writes its lane quarter of TMEM in this CTA, the words of two further
        // groups already on their way, and tells the leader's MMA warp.  Going through TMEM alone, the signal
        // is one that tcgen05.fence orders; words in shared memory would need a release at cluster scope,
        // which beside the loads takes over a microsecond.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
        const uint32_t sf_tmem = tmem + ((uint32_t)(warp & 3) << 21) + 2 * (uint32_t)bt, sf_full0 = mapa(smem_u32(sf_full), 0);
        const int groups = (p.kb + 3) / 4;
        // the group loaded next: tile and its operands, group of K
        int ltile = pair, lq = 0, rows = 0;
        const uint8_t *ws = nullptr, *ts = nullptr;
        auto next = [&](ScaleWords &w) {
            if (ltile >= total) return;
            if (lq == 0) {
                int g, mt, nt;
                pair_coords(p, ltile, g, mt, nt);
                // a weight tile past the matrix's end (the second CTA's) feeds no output: any scale
                const int wb = min(2 * nt + rank, (p.n[g] + BW - 1) / BW - 1), m0 = mt * bt;
                rows = min(bt, p.m - m0);
                ws = p.w_scale[g] + (size_t)wb * p.scale_ld;
                ts = p.a_scale + (size_t)m0 * p.scale_ld;
            }
            load_scales(w, ws, ts, p.scale_ld, rows, lq, lane);
            if (++lq == groups) lq = 0, ltile += pairs;
        };
        ScaleWords w0, w1, w2;
        next(w0);
        next(w1);
        next(w2);
        uint32_t slot = 0, par = 1;
        bool ok = true;
        auto put_group = [&](const ScaleWords &w) {
            __syncwarp();                                // next loads lane by lane
            ok = ok && warp_wait<true>(smem_u32(&sf_empty[slot]), par, abort);
            if (!ok) return;
            fence_after();
            store_scales(sf_tmem + slot * Pair::SF_COLS, w);
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(sf_full0 + 8 * slot);
            __syncwarp();
            if (++slot == SF_SLOTS) slot = 0, par ^= 1;
        };
        const int tiles = pair < total ? (total - pair + pairs - 1) / pairs : 0;
        for (int64_t left = (int64_t)tiles * groups; left > 0 && ok; left -= 3) {
            put_group(w0);
            next(w0);
            if (left > 1) put_group(w1);
            next(w1);
            if (left > 2) put_group(w2);
            next(w2);
        }
        __syncwarp();
    }
    __syncthreads();
    cluster_sync();                                  // the partner's arrivals and MMAs have this CTA's memory until here
    if (warp == 1) {
        // the leader has seen its last commit; that arrives in this CTA's memory too, after all others
        mbar_drain(smem_u32(drain), 0);
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
    }();
    return fn;
}

// Bytes [rows][k] at the quantised pitch, boxes of box_rows x 128 bytes.
cudaError_t make_map(CUtensorMap *map, const uint8_t *p, int64_t rows, int k, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)quant_row_bytes((uint32_t)k)};
    cuuint32_t box[2] = {BK, (cuuint32_t)box_rows}, es[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(p), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tiles of wrows weight rows x bt rows; a CTA loads box_t of the rows at once.
cudaError_t fill_params(const QuantMatmulArgs &a, int wrows, int bt, int box_t, Params &p, Maps &maps) {
    cudaError_t e = make_map(&maps.a, a.a, a.m, a.k, box_t);
    p = Params{};
    p.a_scale = a.a_scale;
    p.m = a.m;
    p.kb = (a.k + BK - 1) / BK;
    p.k_tail = (a.k - (p.kb - 1) * BK + 31) / 32;
    p.scale_ld = (int)quant_scale_bytes((uint32_t)a.k);
    p.m_tiles = (a.m + bt - 1) / bt;
    p.n_w = a.n_w;
    p.bf16_out = a.out_dtype == DS4C_BF16;
    int start = 0;
    for (int g = 0; g < a.n_w && e == cudaSuccess; g++) {
        e = make_map(&maps.w[g], a.w[g].q, a.w[g].n, a.k, BW);
        p.tile_start[g] = start;
        p.n[g] = (int)a.w[g].n;
        p.w_scale[g] = a.w[g].scale;
        p.out[g] = a.w[g].out;
        p.out_ld[g] = (int64_t)a.w[g].out_ld;
        start += (p.n[g] + wrows - 1) / wrows * p.m_tiles;
    }
    p.tile_start[a.n_w] = start;
    for (int g = a.n_w; g < 4; g++) maps.w[g] = maps.w[0];
    return e;
}

// Output tiles of wrows x rows over all weight matrices.
int64_t count_tiles(const QuantMatmulArgs &a, int wrows, int rows) {
    int64_t tiles = 0;
    for (int g = 0; g < a.n_w; g++) tiles += (int64_t)((a.w[g].n + wrows - 1) / wrows) * ((a.m + rows - 1) / rows);
    return tiles;
}

// CTAs that share a tile of bt rows: of 1, 2, 4 and 8 with all clusters running at once, the one with the
// least time of its own (10 ns): 0.33 us a block of K, half as much again and 0.4 us where clusters share
// their SMs, 0.6 us and 11 ns a row for the meeting.  Fitted to 216 products of 1 to 128 rows, 256 to 8192
// columns and K (mean loss to the best choice 0.3 %; as many CTAs as leave each two blocks lost 4.5, 27 at
// most: 128 x 1024 x 512 4.4 us whole and 5.6 by two, 64 x 256 x 1544 4.0 by eight and 5.0 by four).
// Clusters of 2, 4 and 8 CTAs of one SM each that this GPU's 152 SMs hold: 76, 36 and 15 (a cluster stays
// within a group of about 19 SMs); 16 x 8 CTAs took 14.3 us where 16 x 4 take 8.6.
int choose_split(int64_t tiles, int kb, int bt, int per_sm) {
    const int room[4] = {152, 76, 36, 15};
    int split = 1, least = 0;
    for (int i = 0; i < 4; i++) {
        if (i > 0 && (tiles > (int64_t)room[i] * per_sm || kb < 1 << i)) break;
        const int blocks = (kb + (1 << i) - 1) >> i;
        const int cost = (i > 0 ? 60 + 11 * bt / 10 : 0) + (tiles > room[i] ? 40 + 33 * blocks * 3 / 2 : 33 * blocks);
        if (i == 0 || cost < least) split = 1 << i, least = cost;
    }
    return split;
}

template <int BT>
cudaError_t launch_split(const QuantMatmulArgs &a, cudaStream_t s) {
    using S = Shape<BT>;
    Maps maps;
    Params p;
    cudaError_t e = fill_params(a, BW, BT, BT, p, maps);
    if (e != cudaSuccess) return e;
    if ((e = ensure_dyn_smem(qmm_split_kernel<BT>, S::SMEM_BYTES)) != cudaSuccess) return e;
    const int tiles = p.tile_start[a.n_w], split = choose_split(tiles, p.kb, BT, S::PER_SM);
    return launch_pdl_cluster(qmm_split_kernel<BT>, dim3((unsigned)(tiles * split)), dim3(THREADS), S::SMEM_BYTES, s, split,
                              maps, p, split);
}

// Time of the product on split<128>, in 10 ns: 3 us and 0.37 us a block of K for each round of CTAs over the
// SMs, 1.4 us more for meeting in a cluster.
int64_t split_cost(const QuantMatmulArgs &a) {
    const int64_t tiles = count_tiles(a, BW, 128);
    const int kb = (a.k + BK - 1) / BK, split = choose_split(tiles, kb, 128, 1);
    return (tiles * split + 151) / 152 * (300 + 37 * ((kb + split - 1) / split)) + (split > 1 ? 140 : 0);
}

constexpr int PAIRS = 76, JOINT_BT = 160;      // the widest tile whose stages are two blocks of K

// Rows of a pair tile: the width with the fewest rounds over the pairs times a block's time; cost: of the
// product, in 10 ns: 4 us and 0.115 + 0.00058 bt us a block.
int pair_bt(const QuantMatmulArgs &a, int64_t &cost) {
    int best = 0;
    const int kb = (a.k + BK - 1) / BK;
    for (int bt = MAX_BT; bt >= 128; bt -= 32) {
        const int64_t c = 400 + (count_tiles(a, 2 * BW, bt) + PAIRS - 1) / PAIRS * kb * (11500 + 58 * bt) / 1000;
        if (best == 0 || c < cost) best = bt, cost = c;
    }
    return best;
}

__global__ void wait_selftest_kernel(int *answers) {
    warp_wait_selftest(
        answers,
        [](auto look, volatile int *abort) { return warp_bounded_wait<256>(look, abort, g_qmm_wait_ns, &g_qmm_err); },
        [](uint32_t bar, uint32_t parity, volatile int *abort) {
            return warp_wait(bar, parity, abort) && warp_wait<true>(bar, parity, abort);
        });
}

// Whether the warpgroups' registers after setmaxnreg fit what a launch of the pair kernel gives; where they do not, their
// wait for them would never end.  The compiled kernel's register count is asked for until it is known: a failed query is
// the call's error, not an answer.
template <bool joint>
cudaError_t pair_fits(bool &fits) {
    static std::atomic<int> regs{0};
    int n = regs.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, qmm_pair_kernel<joint>);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
        regs.store(n = attr.numRegs, std::memory_order_relaxed);
    }
    fits = 4 * n >= 2 * REG_EPILOGUE + 2 * REG_OTHER;
    return cudaSuccess;
}

cudaError_t launch_pair(const QuantMatmulArgs &a, int bt, cudaStream_t s) {
    Maps maps;
    Params p;
    cudaError_t e = fill_params(a, 2 * BW, bt, bt / 2, p, maps);
    if (e != cudaSuccess) return e;
    auto kernel = bt <= JOINT_BT ? qmm_pair_kernel<true> : qmm_pair_kernel<false>;
    if ((e = ensure_dyn_smem(kernel, Pair::SMEM_BYTES)) != cudaSuccess) return e;
    const int tiles = p.tile_start[a.n_w];
    return launch_pdl(kernel, dim3((unsigned)(2 * (tiles < PAIRS ? tiles : PAIRS))), dim3(PAIR_THREADS), Pair::SMEM_BYTES, s,
                      maps, p, bt);
}

}  // namespace

cudaError_t launch_quant_matmul(const QuantMatmulArgs &a, cudaStream_t s) {
    if (a.m <= 16) return launch_split<16>(a, s);
    if (a.m <= 32) return launch_split<32>(a, s);
    if (a.m <= 64) return launch_split<64>(a, s);
    // more rows: one CTA's tiles, K split to fill the GPU, or pairs' tiles, which reuse more; by the two
    // costs, fitted to 336 products of 96 to 1024 rows with 256 to 8192 columns and K (mean loss to the
    // better one 0.1 %, most 6.5; 256 rows: 4096 x 4096 11.6 us split and 10.9 in pairs, 8192 x 8192 26.1 and
    // 20.5, 1024 x 4096 8.3 and 9.8, 256 x 8192 8.1 and 15.4)
    int64_t cost;
    const int bt = pair_bt(a, cost);
    if (split_cost(a) <= cost) return launch_split<128>(a, s);
    bool fits = false;
    const cudaError_t e = bt <= JOINT_BT ? pair_fits<true>(fits) : pair_fits<false>(fits);
    if (e != cudaSuccess) return e;
    return fits ? launch_pair(a, bt, s) : launch_split<128>(a, s);
}

cudaError_t qmm_wait_selftest(int *answers, cudaStream_t s) {
    wait_selftest_kernel<<<1, 32, 0, s>>>(answers);
    return cudaGetLastError();
}

cudaError_t qmm_set_wait_ns(unsigned long long ns) { return cudaMemcpyToSymbol(g_qmm_wait_ns, &ns, sizeof ns); }

unsigned int qmm_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_qmm_err, sizeof v) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_qmm_err, &z, sizeof z);
    return v;
}

}  // namespace ds4c
