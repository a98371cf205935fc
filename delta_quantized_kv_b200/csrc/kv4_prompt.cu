// kv4_prompt.cu -- prompt attention over the paged 4-bit cache: ragged chunks
// of causal queries, on the 5th-generation tensor cores.
//
// The rows of one kv head are its G query heads of every token, row r of a
// sequence's chunk being token r / G, head r % G; a CTA takes 256 of them as
// two tiles of 128 (the M of one tcgen05.mma) and walks the positions it sees
// in tiles of 128.  Four warpgroups:
//   0, 1   softmax of query tile 0, 1: one thread a row; scores from tensor
//          memory, weights back into it as the A operand of the second product
//   2      dequantisation: one thread a position; packed records from global
//          memory, fp16 values (exact) into swizzled shared memory, two stages
//          each of K and V
//   3      one thread issues every MMA
// Tensor memory: scores S0, S1 (fp32 128 x 128 each, the fp16 weights over
// their first half) and outputs O0, O1.  While the softmax of one query tile
// works, the tensor cores multiply for the other.
//
// A V word holds 8 channels 8 apart, so dequantised words are stored as they
// come: the columns of O are a permutation of the channels, undone in
// registers when O is written.
//
// Softmax, per row: the weights are 2^(x - ref) with ref at least max - 15 and
// at most max - 7 (log2 units); O is rescaled only when the maximum has risen
// by more than 8 since ref was set, so it seldom is.  Weights in [.., 2^15]
// are rounded to fp16 once; sums and scores are fp32.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "kv4_common.cuh"
#include "kv4_internal.h"

namespace dkv {
namespace kv4 {
namespace {

constexpr int TM = 128;            // query rows per tile
constexpr int TN = 128;            // positions per tile
constexpr int THREADS = 640;
constexpr int STAGES = 2;

struct Prompt {
    Query q;
    int G, splits;
    float *ws;                     // splits > 1: [splits][n_rows * Hq][D + 4] partial rows
    int64_t ws_floats;
};

template <int D>
struct Smem {
    static constexpr int SLABS = D / 64;            // 64-channel slabs of 128-byte rows
    static constexpr int TILE = SLABS * 128 * 128;  // bytes of a 128-row fp16 tile
    static constexpr int Q = 0;
    static constexpr int K = 2 * TILE;
    static constexpr int V = K + STAGES * TILE;
    static constexpr int BAR = V + STAGES * TILE;
    static constexpr int END = BAR + 256;
    // one CTA per SM: it takes all of the tensor memory
    static constexpr int BYTES = (END > 120 * 1024 ? END : 120 * 1024) + 1024;
};

// barriers, in 8-byte slots; PFULL: the first and the second half of a tile's
// weights, for each query tile
enum { KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SFULL = 8, PFULL = 10, OFULL = 14, DRAIN = 16,
       N_BAR = 17 };

// ---- tcgen05 ---------------------------------------------------------------
__device__ inline void tm_alloc(uint32_t dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst_smem),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
__device__ inline void tm_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols));
}
// Descriptors come as their low words (the address, and the leading offset);
// HI is the high word.  The k-th step of an operand is a constant further on.
template <uint32_t HI_A, uint32_t HI_B, uint32_t IDESC>
__device__ inline void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %3, 0;\n"
        " mov.b64 da, {%1, %4};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %6, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(acc), "n"(HI_A), "n"(HI_B), "n"(IDESC)
        : "memory");
}
template <uint32_t HI_B, uint32_t IDESC>
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.u32 p, %3, 0;\n"
        " mov.b64 db, {%2, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(acc), "n"(HI_B), "n"(IDESC)
        : "memory");
}
__device__ inline void tm_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(
            smem_u32(bar))
        : "memory");
}
__device__ inline void tm_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ inline void tm_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
#define DKV_RW8(r, i) \
    "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
        "+r"(r[i + 6]), "+r"(r[i + 7])
// Waits for this warp's loads; what uses r comes after.
__device__ inline void tm_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : DKV_RW8(r, 0), DKV_RW8(r, 8), DKV_RW8(r, 16), DKV_RW8(r, 24)::"memory");
}
__device__ inline void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ inline void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

#define DKV_R8(r, i) \
    "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
        "=r"(r[i + 6]), "=r"(r[i + 7])
#define DKV_W8(r, i) \
    "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
        "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this thread's row (lane)
__device__ inline void tm_ld32(uint32_t *r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : DKV_R8(r, 0), DKV_R8(r, 8), DKV_R8(r, 16), DKV_R8(r, 24)
        : "r"(addr));
}
__device__ inline void tm_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
        DKV_W8(r, 0), DKV_W8(r, 8), DKV_W8(r, 16), DKV_W8(r, 24)
        : "memory");
}
__device__ inline void tm_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};\n" ::"r"(addr),
        DKV_W8(r, 0), DKV_W8(r, 8)
        : "memory");
}

// A bounded wait whose outcome the whole warp shares.
__device__ inline bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}
// Registers of this warpgroup.  640 threads are launched with 96 each; 2 x 152
// + 2 x 64 + 48 = 5 x 96.
template <int N>
__device__ inline void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ inline void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

__device__ inline void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// One arrival for the warp, behind what all its lanes did.
__device__ inline void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Instruction descriptor, kind::f16: fp16 A and B, fp32 D, A K-major.
__device__ constexpr uint32_t idesc(int m, int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle: low word from the address and the
// leading offset, high word from the stride offset (all in bytes).
__device__ inline uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
    return ((addr >> 4) & 0x3FFFu) | (lbo >> 4) << 16;
}
__device__ constexpr uint32_t desc_hi(uint32_t sbo) { return sbo >> 4 | 1u << 14 | 2u << 29; }
__device__ inline bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ inline float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ inline uint64_t f2(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ inline float f2_lo(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ inline float f2_hi(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ inline uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// 2^x of two x on the FMA pipes (-126 <= x < 127, finite; below, 2^-126): x = n
// + f with |f| <= 1/2 by adding 1.5 * 2^23, and 2^f by the degree-5 polynomial
// of least relative error with p(0) = 1.  Error 1.6e-7, below ex2.approx's.
__device__ inline uint64_t ex2_poly(uint64_t x) {
    x = f2(fmaxf(f2_lo(x), -126.f), fmaxf(f2_hi(x), -126.f));
    const uint64_t t = add2(x, f2(12582912.f, 12582912.f));
    const uint64_t n = add2(t, f2(-12582912.f, -12582912.f));
    const uint64_t f = fma2(n, f2(-1.f, -1.f), x);
    uint64_t y = f2(0x1.5bba14p-10f, 0x1.5bba14p-10f);
    y = fma2(y, f, f2(0x1.3cea88p-7f, 0x1.3cea88p-7f));
    y = fma2(y, f, f2(0x1.c6b752p-5f, 0x1.c6b752p-5f));
    y = fma2(y, f, f2(0x1.ebf9bcp-3f, 0x1.ebf9bcp-3f));
    y = fma2(y, f, f2(0x1.62e42ap-1f, 0x1.62e42ap-1f));
    y = fma2(y, f, f2(1.f, 1.f));
    return (uint64_t)((uint32_t)(y >> 32) + ((uint32_t)(t >> 32) << 23)) << 32 |
           (uint64_t)((uint32_t)y + ((uint32_t)t << 23));
}

// Exponent e with max |q| 2^e in [2^14, 2^15).
__device__ inline int q_exponent(float mx) {
    if (!(mx > 0.f)) return 0;
    const int e = 14 - (int)((__float_as_uint(mx) >> 23) & 255u) + 127;
    return max(-100, min(120, e));
}

// The work of one CTA.
struct Job {
    int b, kvh;
    int row0, nrow;        // first row of the 256, rows of the sequence's chunk (tokens * G)
    int tok0;              // first token row of the sequence in Q
    int pos0;              // position of the chunk's first token
    int kv0, ntile;        // first position of tile 0; position tiles
    int len;
};

// Finds the CTA's job; false if it has none.  A whole warp asks.
__device__ inline bool find_job(const View &v, const Prompt &p, int x, int split, Job *j) {
    const int lane = threadIdx.x & 31;
    j->kvh = x % v.H;
    const int want = x / v.H;
    // blocks of 256 rows of a sequence
    auto blocks = [&](int b, int *n_out) {
        *n_out = 0;
        if (b >= v.B) return 0;
        const int s0 = seq_start(v, b);
        const int n = (v.starts ? v.starts[b + 1] : s0 + v.n_uniform) - s0;
        if (n <= 0 || s0 < 0) return 0;
        const int len = seq_len(v, b);
        if (len < 0) return 0;
        if (n > len || s0 + n > v.n_rows) {      // more rows than positions or queries
            set_status(v.status, DKV_DEV_BAD_SEQLEN);
            return 0;
        }
        *n_out = n;
        return (int)(((int64_t)n * p.G + 2 * TM - 1) / (2 * TM));
    };
    int n, total = 0;
    for (int b0 = 0; b0 < v.B; b0 += 32) {
        int k = blocks(b0 + lane, &n);
#pragma unroll
        for (int o = 16; o; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
        total += k;
    }
    // the last blocks, which see most, first
    int left = total - 1 - want;
    if (left < 0) return false;
    for (int b0 = 0; b0 < v.B; b0 += 32) {
        const int k = blocks(b0 + lane, &n);
        int inc = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left);
        if (hit) {
            const int l = __ffs(hit) - 1;
            left -= __shfl_sync(0xffffffffu, inc - k, l);
            n = __shfl_sync(0xffffffffu, n, l);
            j->b = b0 + l;
            j->row0 = left * 2 * TM;
            j->nrow = n * p.G;
            j->tok0 = seq_start(v, j->b);
            j->len = v.lens[j->b];
            j->pos0 = j->len - n;
            const int first = j->pos0 + j->row0 / p.G;
            const int last = j->pos0 + (min(j->row0 + 2 * TM, j->nrow) - 1) / p.G;
            int lo = p.q.window > 0 ? max(0, first - p.q.window + 1) : 0;
            lo &= ~(RT - 1);
            const int tiles = (last + 1 - lo + TN - 1) / TN;
            // this split's share
            const int t0 = (int)((int64_t)tiles * split / p.splits);
            const int t1 = (int)((int64_t)tiles * (split + 1) / p.splits);
            j->kv0 = lo + t0 * TN;
            j->ntile = t1 - t0;
            return true;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// 8 codes of word w -> 8 fp16 values in nibble order 0,4,1,5,2,6,3,7.
// z1024 = 1024 + zero, z64 = 64 + zero in both halves.
__device__ inline uint4 dequant8(uint32_t w, __half2 s, __half2 z1024, __half2 z64) {
    const uint32_t w8 = w >> 8;
    uint32_t a, b, c, d;
    a = and_or<0x000F000Fu>(w, 0x64006400u);
    b = and_or<0x00F000F0u>(w, 0x54005400u);
    c = and_or<0x000F000Fu>(w8, 0x64006400u);
    d = and_or<0x00F000F0u>(w8, 0x54005400u);
    return make_uint4(h2_as_u32(__hmul2(__hsub2(u32_as_h2(a), z1024), s)),
                      h2_as_u32(__hmul2(__hsub2(u32_as_h2(b), z64), s)),
                      h2_as_u32(__hmul2(__hsub2(u32_as_h2(c), z1024), s)),
                      h2_as_u32(__hmul2(__hsub2(u32_as_h2(d), z64), s)));
}

struct Meta {
    __half2 s, z1024, z64;
};
__device__ inline Meta meta_of(uint32_t m) {       // one block's halfword
    Meta r;
    const uint32_t mm = m | m << 16;
    r.s = meta_scale(mm);
    r.z1024 = u32_as_h2(and_or<0x000F000Fu>(mm, 0x64006400u));
    r.z64 = u32_as_h2(((mm << 4) & 0x00F000F0u) | 0x54005400u);
    return r;
}

// Bits below n.
__device__ inline uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// Scores that the row does not see.
__device__ inline void hide(uint32_t (&s)[32], uint32_t see) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (!(see >> k & 1)) s[k] = 0xFF800000u;
}
__device__ inline float max32(const uint32_t (&s)[32]) {
    float a = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    float b = fmaxf(__uint_as_float(s[2]), __uint_as_float(s[3]));
#pragma unroll
    for (int k = 4; k < 32; k += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
        b = fmaxf(fmaxf(b, __uint_as_float(s[k + 2])), __uint_as_float(s[k + 3]));
    }
    return fmaxf(a, b);
}

// 32 of a row's scores to weights 2^(c s + r), as fp16 and into the sum.  NP of
// the 16 pairs go by the polynomial, the others by ex2.approx: that unit gives
// 16 results a clock and SM, 2048 clocks for the CTA's two tiles, as long as
// the tensor cores take.
constexpr int POLY = 4;
template <int NP>
__device__ inline void weights(const uint32_t (&s)[32], uint64_t c2, uint64_t r2,
                               uint32_t (&w)[16], uint64_t &l2) {
    uint64_t la = l2, lb = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint64_t x = fma2((uint64_t)s[2 * k + 1] << 32 | s[2 * k], c2, r2);
        uint64_t y;
        if (NP > 0 && (k * NP) % 16 < NP) y = ex2_poly(x);
        else y = f2(ex2(f2_lo(x)), ex2(f2_hi(x)));
        if (k & 1) lb = add2(lb, y);
        else la = add2(la, y);
        w[k] = pack_h2(f2_lo(y), f2_hi(y));
    }
    l2 = add2(la, lb);
}

template <typename L, int DT>
__global__ void __launch_bounds__(THREADS, 1)
prompt_kernel(View v, Prompt p) {
    using S = Smem<L::D>;
    extern __shared__ uint8_t smem_raw[];
    // descriptors want 1024-byte atoms
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::BAR);
    uint32_t *tm_slot = reinterpret_cast<uint32_t *>(smem + S::BAR + N_BAR * 8);
    // [4]: records of a position tile that are there, 2 bits in each byte (by
    // dequantising warp).  Tile j + 4's is written after tile j + 1's weights
    // have been multiplied, so after tile j's was read.
    volatile uint32_t *valid = tm_slot + 1;
    constexpr uint32_t ALL = 0x03030303u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    const int tid = threadIdx.x & 127;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bars + KFULL + i, 4);
            mbar_init(bars + KFREE + i, 1);
            mbar_init(bars + VFULL + i, 4);
            mbar_init(bars + VFREE + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + SFULL + i, 1);
            mbar_init(bars + PFULL + 2 * i, 4);
            mbar_init(bars + PFULL + 2 * i + 1, 4);
            mbar_init(bars + OFULL + i, 1);
        }
        mbar_init(bars + DRAIN, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    Job job;
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) check_starts(v);
    if (!find_job(v, p, blockIdx.x, blockIdx.y, &job)) return;    // all warps agree
    if (warp == 16) tm_alloc(smem_u32(tm_slot), 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tm = *tm_slot;
    const int ntile = job.ntile;
    const int qtiles = job.nrow - job.row0 > TM ? 2 : 1;

    if (wg < 2) {
        // ---------------- softmax ------------------------------------------
        regs_up<152>();
        const int qi = wg;
        const int row = job.row0 + qi * TM + tid;
        const bool have = row < job.nrow;
        const int tok = have ? row / p.G : 0, head = job.kvh * p.G + (have ? row - tok * p.G : 0);
        const int pos = have ? job.pos0 + tok : -1;
        const int lo = p.q.window > 0 ? pos - p.q.window : -1;        // sees (lo, pos]
        float c1 = p.q.scale * 1.44269504088896340736f;
        bool ok = true;
        if (qi < qtiles) {
            // the row's query into the swizzled tile
            uint8_t *qrow = smem + S::Q + qi * S::TILE + tid * 128;
            const uint16_t *src = static_cast<const uint16_t *>(p.q.q) +
                                  (int64_t)(job.tok0 + tok) * p.q.tok + (int64_t)head * p.q.head;
            uint4 u[L::D / 8];
#pragma unroll
            for (int i = 0; i < L::D / 8; ++i)
                u[i] = have ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
            if constexpr (DT == DKV_BF16) {
                // bf16 as fp16, by a power of two: exact down to 2^-28 of the
                // row's largest
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < L::D / 8; ++i) {
                    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                             fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
                }
                const int e = q_exponent(mx);
                const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                c1 *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < L::D / 8; ++i) {
                    uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_h2(__uint_as_float(w[k] << 16) * up,
                                       __uint_as_float(w[k] & 0xFFFF0000u) * up);
                    u[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < L::D / 8; ++i)
                *reinterpret_cast<uint4 *>(qrow + (i >> 3) * (128 * 128) +
                                           (((i & 7) ^ (tid & 7)) << 4)) = u[i];
        }
        fence_proxy_async();
        // both query tiles are in place before the first MMA
        asm volatile("bar.sync 1, 288;\n" ::: "memory");       // 8 softmax warps + the MMA warp
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
        const uint32_t tS = tm + lane_base + qi * 128, tO = tm + lane_base + 256 + qi * L::D;
        float ref = 0.f;
        uint64_t l2 = 0;                   // the sum, in two halves
        bool any = false;                  // ref has been set
        const int row_first = job.row0 + qi * TM;
        const int pmin = job.pos0 + row_first / p.G;     // the tile's first and last positions
        const int pmax = job.pos0 + (min(row_first + TM, job.nrow) - 1) / p.G;
        if (qi < qtiles) {
            for (int j = 0; j < ntile; ++j) {
                if (!warp_wait(bars + SFULL + qi, j & 1)) { ok = false; break; }
                tm_fence_after();
                // all scores are looked at for the maximum, then the second half is
                // loaded again: 128 of them do not stay in registers
                uint32_t s0[32], s1[32];
                const int kv = job.kv0 + j * TN;
                const uint32_t vm = valid[j & 3];
                const bool edge = kv + TN - 1 > pmin ||
                                  (p.q.window > 0 && kv <= pmax - p.q.window) || vm != ALL;
                // (the row sees (lo, pos], and records that are there)
                auto see = [&](int i) {
                    const int at = kv + 32 * i;
                    const uint32_t v2 = vm >> (8 * i);
                    return below(pos + 1 - at) & ~below(lo + 1 - at) &
                           ((v2 & 1 ? 0xFFFFu : 0u) | (v2 & 2 ? 0xFFFF0000u : 0u));
                };
                float mx;
                {
                    uint32_t s2[32], s3[32];
                    tm_ld32(s0, tS);
                    tm_ld32(s1, tS + 32);
                    tm_ld32(s2, tS + 64);
                    tm_ld32(s3, tS + 96);
                    tm_wait_ld32(s0);
                    tm_wait_ld32(s1);
                    tm_wait_ld32(s2);
                    tm_wait_ld32(s3);
                    if (edge) {
                        hide(s0, see(0));
                        hide(s1, see(1));
                        hide(s2, see(2));
                        hide(s3, see(3));
                    }
                    mx = fmaxf(fmaxf(max32(s0), max32(s1)), fmaxf(max32(s2), max32(s3))) * c1;
                }
                // (NaN scores leave mx to the others; their weights are NaN)
                const bool up = mx > -INFINITY && (!any || mx > ref + 15.f);
                if (__any_sync(0xffffffffu, up)) {
                    const float nref = up ? mx - 7.f : ref;
                    const float f = any ? ex2(ref - nref) : 0.f;
                    if (j > 0) {
                        // O must be at rest
                        if (!warp_wait(bars + OFULL + qi, (j - 1) & 1)) { ok = false; break; }
                        tm_fence_after();
#pragma unroll
                        for (int i = 0; i < L::D / 32; ++i) {
                            uint32_t o[32];
                            tm_ld32(o, tO + 32 * i);
                            tm_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(up ? __uint_as_float(o[k]) * f
                                                          : __uint_as_float(o[k]));
                            tm_st32(tO + 32 * i, o);
                        }
                    }
                    if (up) {
                        l2 = fma2(l2, f2(f, f), 0);
                        ref = nref;
                        any = true;
                    }
                }
                // the polynomial takes finite scores only
                const uint64_t c2 = f2(c1, c1), r2 = f2(-ref, -ref);
                const bool plain = edge || !__all_sync(0xffffffffu, fabsf(mx) < INFINITY);
                uint32_t w[16];
                auto put = [&](int i, uint32_t (&s)[32]) {
                    if (plain) weights<0>(s, c2, r2, w, l2);
                    else weights<POLY>(s, c2, r2, w, l2);
                    tm_st16(tS + 16 * i, w);
                    if (i & 1) {
                        tm_wait_st();
                        tm_fence_before();
                        warp_arrive(bars + PFULL + 2 * qi + (i >> 1));
                    }
                };
                put(0, s0);
                tm_ld32(s0, tS + 64);
                put(1, s1);
                tm_ld32(s1, tS + 96);
                tm_wait_ld32(s0);
                tm_wait_ld32(s1);
                if (edge) {
                    hide(s0, see(2));
                    hide(s1, see(3));
                }
                put(2, s0);
                put(3, s1);
            }
            const float l = f2_lo(l2) + f2_hi(l2);
            // ---------------- output ---------------------------------------
            if (ok && ntile > 0) ok = warp_wait(bars + OFULL + qi, (ntile - 1) & 1);
            if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
            tm_fence_after();
            const int64_t orow = (int64_t)(job.tok0 + tok) * p.q.Hq + head;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);       // NaN stays NaN
            float *part = p.splits > 1
                              ? p.ws + ((int64_t)blockIdx.y * v.n_rows * p.q.Hq + orow) * (L::D + 4)
                              : nullptr;
#pragma unroll
            for (int u = 0; u < L::D / 64; ++u) {
                uint32_t o[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) o[i] = 0;
                if (ntile > 0) {
                    tm_ld32(o, tO + 64 * u);
                    tm_ld32(o + 32, tO + 64 * u + 32);
                    tm_wait_ld();
                }
                if (!have) continue;
                // column 64 u + 8 g + at(n) is channel 64 u + 8 n + g (n: nibble)
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int at = n < 4 ? 2 * n : 2 * (n - 4) + 1;
                    float y[8];
#pragma unroll
                    for (int g = 0; g < 8; ++g) y[g] = __uint_as_float(o[8 * g + at]) * inv;
                    const int ch = 64 * u + 8 * n;
                    if (part) {
                        if (range_ok(v.status, part + ch, 32, p.ws, p.ws_floats * 4)) {
                            reinterpret_cast<float4 *>(part + ch)[0] =
                                make_float4(y[0], y[1], y[2], y[3]);
                            reinterpret_cast<float4 *>(part + ch)[1] =
                                make_float4(y[4], y[5], y[6], y[7]);
                        }
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (DT == DKV_F16) {
                                w[k] = pack_h2(y[2 * k], y[2 * k + 1]);
                            } else {
                                const __nv_bfloat162 h =
                                    __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
                                w[k] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                        }
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.q.out) +
                                                   orow * L::D + ch) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (have) {
                if (part) {
                    if (range_ok(v.status, part + L::D, 8, p.ws, p.ws_floats * 4)) {
                        part[L::D] = any ? ref : -INFINITY;
                        part[L::D + 1] = l;
                    }
                } else if (p.q.lse) {
                    p.q.lse[orow] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994530942f;
                }
            }
        }
    } else if (wg < 4) {
        // ---------------- dequantisation: K (2), V (3) ---------------------
        regs_down<64>();
        bool ok = true;
        const bool isk = wg == 2;
        uint64_t *full = bars + (isk ? KFULL : VFULL), *free_ = bars + (isk ? KFREE : VFREE);
        uint32_t cw[L::D / 8], cm[L::NB], nw[L::D / 8], nm[L::NB];
        bool here = false;
        // position `at`'s words; false where the record is missing below the
        // length (a bad page): it is not seen
        auto fetch = [&](int j) {
            const int at = job.kv0 + j * TN + tid;
            const uint8_t *rec = at < job.len ? record(v, job.b, job.kvh, at, L::REC) : nullptr;
            if (rec && !range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes))
                rec = nullptr;
            const int t = at & (RT - 1);
#pragma unroll
            for (int i = 0; i < L::D / 8; ++i) nw[i] = 0u;
#pragma unroll
            for (int i = 0; i < L::NB; ++i) nm[i] = 0u;
            if (rec) {
                const uint4 *a = reinterpret_cast<const uint4 *>(
                    rec + (isk ? L::k_word(t, 0) : L::OFF_V + t * L::ROW));
#pragma unroll
                for (int i = 0; i < L::D / 32; ++i) {
                    const uint4 x = a[i];
                    nw[4 * i] = x.x; nw[4 * i + 1] = x.y; nw[4 * i + 2] = x.z; nw[4 * i + 3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < L::NB; ++i)
                    nm[i] = *reinterpret_cast<const uint16_t *>(
                        rec + (isk ? L::k_meta(t, i) : L::v_meta(t, i)));
            }
            here = rec != nullptr || at >= job.len;
        };
        if (ntile > 0) fetch(0);
        for (int j = 0; j < ntile; ++j) {
            const int st = j % STAGES, ph = (j / STAGES) & 1;
#pragma unroll
            for (int i = 0; i < L::D / 8; ++i) cw[i] = nw[i];
#pragma unroll
            for (int i = 0; i < L::NB; ++i) cm[i] = nm[i];
            const unsigned there = __ballot_sync(0xffffffffu, here);
            if (j + 1 < ntile) fetch(j + 1);
            if (j >= STAGES && !warp_wait(free_ + st, ph ^ 1)) { ok = false; break; }
            Meta m[L::NB];
#pragma unroll
            for (int i = 0; i < L::NB; ++i) m[i] = meta_of(cm[i]);
            uint8_t *dst = smem + (isk ? S::K : S::V) + st * S::TILE + tid * 128;
            if (isk) {
                if (lane == 0)          // two records a warp: lanes 0..15 and 16..31
                    reinterpret_cast<volatile uint8_t *>(valid + (j & 3))[warp & 3] =
                        (uint8_t)(((there & 0xFFFFu) == 0xFFFFu ? 1 : 0) |
                                  ((there >> 16) == 0xFFFFu ? 2 : 0));
#pragma unroll
                for (int w = 0; w < L::D / 8; ++w) {
                    const int c8 = 4 * (w % L::NJ) + w / L::NJ;       // word t * NJ + j
                    const Meta &q = m[c8 * 8 / L::G];
                    *reinterpret_cast<uint4 *>(dst + (c8 >> 3) * (128 * 128) +
                                               (((c8 & 7) ^ (tid & 7)) << 4)) =
                        dequant8(cw[w], q.s, q.z1024, q.z64);
                }
            } else {
                const int t = (job.kv0 + j * TN + tid) & (RT - 1);
                const int flip = L::D == 128 ? ((t >> 1) & 1) << 2 : 0;
#pragma unroll
                for (int w = 0; w < L::D / 8; ++w) {
                    // D = 128: words 2 c + u of chunk position c = g ^ flip; the word's
                    // nibbles are channels 16 mt + 8 e + g, mt = 4 u ..: two blocks of
                    // 32 channels (nibbles 0-3 and 4-7), or one of 64
                    const int c = L::D == 128 ? w >> 1 : w, u = L::D == 128 ? w & 1 : 0;
                    const int g = c ^ flip;
                    uint4 y;
                    if constexpr (L::G == 64) {
                        y = dequant8(cw[w], m[u].s, m[u].z1024, m[u].z64);
                    } else {
                        // low halves are nibbles 0-3, high halves 4-7
                        const Meta &a = m[2 * u], &b = m[2 * u + 1];
                        y = dequant8(cw[w], __lows2half2(a.s, b.s), __lows2half2(a.z1024, b.z1024),
                                     __lows2half2(a.z64, b.z64));
                    }
                    *reinterpret_cast<uint4 *>(dst + u * (128 * 128) +
                                               ((g ^ (tid & 7)) << 4)) = y;
                }
            }
            fence_proxy_async();
            warp_arrive(full + st);
        }
        if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
    } else {
        // ---------------- MMA ----------------------------------------------
        // the warp walks in step, one thread of it issues: everything the
        // instructions take is the same in all lanes
        regs_down<48>();
        if (warp == 16) {
            asm volatile("bar.sync 1, 288;\n" ::: "memory");
            bool ok = true;
            constexpr uint32_t IS = idesc(TM, TN, false), IO = idesc(TM, L::D, true);
            constexpr uint32_t HI = desc_hi(1024);
            const bool leader = elect_one();
            const uint32_t q0 = desc_lo(smem_u32(smem + S::Q), 16),
                           k0 = desc_lo(smem_u32(smem + S::K), 16),
                           v0 = desc_lo(smem_u32(smem + S::V), 128 * 128);
            auto scores = [&](int qi, int st) {
                const uint32_t a = q0 + qi * (S::TILE >> 4), b = k0 + st * (S::TILE >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < L::D / 16; ++k) {
                        const uint32_t off = (k >> 2) * (128 * 128 >> 4) + (k & 3) * (32 >> 4);
                        mma_ss<HI, HI, IS>(tm + qi * 128, a + off, b + off, k > 0);
                    }
                    tm_commit(bars + SFULL + qi);
                }
                __syncwarp();
            };
            auto values = [&](int qi, int st, int half, bool acc) {
                const uint32_t a = tm + qi * 128 + half * (TN / 4);
                const uint32_t b = v0 + (st * S::TILE + half * (TN / 32) * 2048 >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < TN / 32; ++k)
                        mma_ts<HI, IO>(tm + 256 + qi * L::D, a + k * 8, b + k * (2048 >> 4),
                                       acc || k > 0);
                    if (half) tm_commit(bars + OFULL + qi);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t *bar) {
                if (leader) tm_commit(bar);
                __syncwarp();
            };
            if (ntile > 0) {
                ok = warp_wait(bars + KFULL, 0);
                tm_fence_after();
                if (ok) {
                    for (int qi = 0; qi < qtiles; ++qi) scores(qi, 0);
                    commit(bars + KFREE);
                }
            }
            for (int j = 0; ok && j < ntile; ++j) {
                const int st = j % STAGES, ph = (j / STAGES) & 1;
                const int sn = (j + 1) % STAGES, pn = ((j + 1) / STAGES) & 1;
                ok = warp_wait(bars + VFULL + st, ph);
                if (!ok) break;
                for (int qi = 0; qi < qtiles; ++qi) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && warp_wait(bars + PFULL + 2 * qi + half, j & 1);
                        tm_fence_after();
                        if (ok) values(qi, st, half, j > 0 || half > 0);
                    }
                    if (!ok) break;
                    if (j + 1 < ntile) {
                        if (qi == 0) {
                            ok = warp_wait(bars + KFULL + sn, pn);
                            if (!ok) break;
                            tm_fence_after();
                        }
                        scores(qi, sn);
                    }
                }
                if (!ok) break;
                commit(bars + VFREE + st);
                if (j + 1 < ntile) commit(bars + KFREE + sn);
            }
            if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
            // nothing is in flight when tensor memory is given back
            commit(bars + DRAIN);
            warp_wait(bars + DRAIN, 0);
        }
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 16) tm_free(tm, 512);
}

// Joins the splits of a row: one warp per (row, head).
template <int D, int DT>
__global__ void __launch_bounds__(128)
join_kernel(View v, Prompt p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)v.n_rows * p.q.Hq;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= rows) return;
    // only rows that a job wrote: those of a sequence that is in order
    const int tok = (int)(r / p.q.Hq);
    const int b = find_seq(v, tok);
    if (b >= v.B) return;
    const int s0 = seq_start(v, b);
    const int n = (v.starts ? v.starts[b + 1] : s0 + v.n_uniform) - s0;
    if (n <= 0 || s0 < 0 || tok < s0 || tok >= s0 + n || s0 + n > v.n_rows) return;
    const int len = seq_len(v, b);
    if (len < 0 || n > len) return;
    constexpr int W = D / 32;
    float m = -INFINITY, l = 0.f, o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = 0.f;
    for (int s = 0; s < p.splits; ++s) {
        const float *x = p.ws + ((int64_t)s * rows + r) * (D + 4);
        if (!range_ok(v.status, x, (D + 4) * 4, p.ws, p.ws_floats * 4)) return;
        const float ms = x[D], ls = x[D + 1];
        const float mx = fmaxf(m, ms), ref = mx == -INFINITY ? 0.f : mx;
        const float f0 = ex2(m - ref), f1 = ex2(ms - ref) * ls;     // the parts are normalised
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = fmaf(o[i], f0, x[lane * W + i] * f1);
        l = fmaf(l, f0, f1);
        m = mx;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        if constexpr (DT == DKV_F16) {
            w[i] = pack_h2(o[2 * i] * inv, o[2 * i + 1] * inv);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.q.out) + r * D) +
                    lane * (W / 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) dst[i] = w[i];
    if (p.q.lse && lane == 0)
        p.q.lse[r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

constexpr int kMaxDevices = 64;

cudaError_t sm_count(int *n) {
    static std::mutex mu;
    static int known[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {
        e = cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    *n = known[dev];
    return cudaSuccess;
}

// Blocks of 256 rows that the batch may have, and the splits of their
// positions: enough CTAs for the GPU when there are few rows, none of them with
// less than four position tiles at the table's capacity.
struct Grid {
    int64_t blocks;
    int splits;
};
cudaError_t grid_of(const View &v, int Hq, bool ragged, Grid *g) {
    const int G = Hq / v.H;
    g->blocks = ((int64_t)v.n_rows * G + 2 * TM - 1) / (2 * TM);
    if (ragged) {                         // every sequence may end inside a block
        const int64_t most = v.B < v.n_rows ? v.B : v.n_rows;
        g->blocks += most;
    } else {
        g->blocks = (int64_t)v.B * (((int64_t)(v.n_rows / v.B) * G + 2 * TM - 1) / (2 * TM));
    }
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t cap = (int64_t)v.max_pages * v.page_size / (4 * TN);
    int64_t s = sms / (g->blocks * v.H);
    s = s < cap ? s : cap;
    g->splits = (int)(s < 1 ? 1 : (s > 32 ? 32 : s));
    return cudaSuccess;
}

template <typename L, int DT>
cudaError_t launch(const View &v, const Prompt &p, int64_t blocks, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(prompt_kernel<L, DT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<L::D>::BYTES);
    if (e == cudaSuccess)
        e = launch_pdl(prompt_kernel<L, DT>, dim3((unsigned)(blocks * v.H), p.splits),
                       dim3(THREADS), Smem<L::D>::BYTES, st, v, p);
    if (e == cudaSuccess && p.splits > 1)
        e = launch_pdl(join_kernel<L::D, DT>,
                       dim3((unsigned)(((int64_t)v.n_rows * p.q.Hq + 3) / 4)), dim3(128), 0, st, v,
                       p);
    return e;
}
template <typename L>
cudaError_t launch_dt(const View &v, const Prompt &p, int64_t blocks, cudaStream_t st) {
    return p.q.dtype == DKV_F16 ? launch<L, DKV_F16>(v, p, blocks, st)
                                : launch<L, DKV_BF16>(v, p, blocks, st);
}

}  // namespace

cudaError_t prompt_workspace_floats(const View &v, int D, int Hq, bool ragged, int64_t *floats) {
    Grid g;
    const cudaError_t e = grid_of(v, Hq, ragged, &g);
    if (e != cudaSuccess) return e;
    *floats = g.splits > 1 ? (int64_t)g.splits * v.n_rows * Hq * (D + 4) : 4;
    return cudaSuccess;
}

cudaError_t launch_prompt(const View &v, int D, int G, const Query &q, float *ws,
                          int64_t ws_floats, cudaStream_t st) {
    Grid g;
    const cudaError_t e = grid_of(v, q.Hq, v.starts != nullptr, &g);
    if (e != cudaSuccess) return e;
    Prompt p;
    p.q = q;
    p.G = q.Hq / v.H;
    p.splits = g.splits;
    p.ws = ws;
    p.ws_floats = ws_floats;
    if (D == 128)
        return G == 32 ? launch_dt<Lay<128, 32>>(v, p, g.blocks, st)
                       : launch_dt<Lay<128, 64>>(v, p, g.blocks, st);
    return G == 32 ? launch_dt<Lay<64, 32>>(v, p, g.blocks, st)
                   : launch_dt<Lay<64, 64>>(v, p, g.blocks, st);
}

}  // namespace kv4
}  // namespace dkv
