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
constexpr int THREADS = 512;
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

// barriers, in 8-byte slots
enum { KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SFULL = 8, PFULL = 10, OFULL = 12, DRAIN = 14,
       N_BAR = 15 };

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
__device__ inline void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
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
// Registers of this warpgroup.  512 threads are launched with 128 each; 2 x 184
// + 96 + 40 <= 4 x 128.
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

// Instruction descriptor, kind::f16: fp16 A and B, fp32 D, A K-major.
__device__ constexpr uint32_t idesc(int m, int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle: leading and stride byte offsets.
__device__ inline uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ inline float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
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
            mbar_init(bars + KFULL + i, 128);
            mbar_init(bars + KFREE + i, 1);
            mbar_init(bars + VFULL + i, 128);
            mbar_init(bars + VFREE + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + SFULL + i, 1);
            mbar_init(bars + PFULL + i, 128);
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
    if (warp == 12) tm_alloc(smem_u32(tm_slot), 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tm = *tm_slot;
    const int ntile = job.ntile;
    const int qtiles = job.nrow - job.row0 > TM ? 2 : 1;

    if (wg < 2) {
        // ---------------- softmax ------------------------------------------
        regs_up<184>();
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
        float ref = 0.f, l = 0.f;
        bool any = false;                  // ref has been set
        const int row_first = job.row0 + qi * TM;
        const int pmin = job.pos0 + row_first / p.G;     // the tile's first and last positions
        const int pmax = job.pos0 + (min(row_first + TM, job.nrow) - 1) / p.G;
        if (qi < qtiles) {
            for (int j = 0; j < ntile; ++j) {
                if (!warp_wait(bars + SFULL + qi, j & 1)) { ok = false; break; }
                tm_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int i = 0; i < 4; ++i) tm_ld32(s + 32 * i, tS + 32 * i);
                tm_wait_ld();
                const int kv = job.kv0 + j * TN;
                const uint32_t vm = valid[j & 3];
                if (kv + TN - 1 > pmin || (p.q.window > 0 && kv <= pmax - p.q.window) ||
                    vm != ALL) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) {
                        const int at = kv + i;
                        if (at > pos || at <= lo || !(vm >> (i / 32 * 8 + i / RT % 2) & 1)) s[i] = 0xFF800000u;
                    }
                }
                float mx = __uint_as_float(s[0]);
#pragma unroll
                for (int i = 1; i < 127; i += 2)
                    mx = fmaxf(fmaxf(mx, __uint_as_float(s[i])), __uint_as_float(s[i + 1]));
                mx = fmaxf(mx, __uint_as_float(s[127])) * c1;
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
                        l *= f;
                        ref = nref;
                        any = true;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float a = ex2(fmaf(__uint_as_float(s[32 * i + 2 * k]), c1, -ref));
                        const float b = ex2(fmaf(__uint_as_float(s[32 * i + 2 * k + 1]), c1, -ref));
                        l += a + b;
                        w[k] = pack_h2(a, b);
                    }
                    tm_st16(tS + 16 * i, w);
                }
                tm_wait_st();
                tm_fence_before();
                mbar_arrive(bars + PFULL + qi);
            }
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
    } else if (wg == 2) {
        regs_down<96>();
        // ---------------- dequantisation -----------------------------------
        bool ok = true;
        uint32_t kw[L::D / 8], vw[L::D / 8], km[L::NB], vmeta[L::NB];
        const uint32_t sw = (uint32_t)tid * 128u;
        auto fetch = [&](int j) {
            const int at = job.kv0 + j * TN + tid;
            const uint8_t *rec = at < job.len ? record(v, job.b, job.kvh, at, L::REC) : nullptr;
            if (rec && !range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes))
                rec = nullptr;
            const int t = at & (RT - 1);
#pragma unroll
            for (int i = 0; i < L::D / 8; ++i) kw[i] = vw[i] = 0u;
#pragma unroll
            for (int i = 0; i < L::NB; ++i) km[i] = vmeta[i] = 0u;
            if (rec) {
                const uint4 *a = reinterpret_cast<const uint4 *>(rec + L::k_word(t, 0));
                const uint4 *b = reinterpret_cast<const uint4 *>(rec + L::OFF_V + t * L::ROW);
#pragma unroll
                for (int i = 0; i < L::D / 32; ++i) {
                    const uint4 x = a[i], y = b[i];
                    kw[4 * i] = x.x; kw[4 * i + 1] = x.y; kw[4 * i + 2] = x.z; kw[4 * i + 3] = x.w;
                    vw[4 * i] = y.x; vw[4 * i + 1] = y.y; vw[4 * i + 2] = y.z; vw[4 * i + 3] = y.w;
                }
#pragma unroll
                for (int i = 0; i < L::NB; ++i) {
                    km[i] = *reinterpret_cast<const uint16_t *>(rec + L::k_meta(t, i));
                    vmeta[i] = *reinterpret_cast<const uint16_t *>(rec + L::v_meta(t, i));
                }
            }
            // a record that is missing below the length (a bad page) is not seen
            return (unsigned)__ballot_sync(0xffffffffu, rec != nullptr || at >= job.len);
        };
        unsigned there = ntile > 0 ? fetch(0) : 0u;
        for (int j = 0; j < ntile; ++j) {
            const int st = j % STAGES, ph = (j / STAGES) & 1;
            // K
            if (j >= STAGES && !warp_wait(bars + KFREE + st, ph ^ 1)) { ok = false; break; }
            if (lane == 0)          // two records a warp: lanes 0..15 and 16..31
                reinterpret_cast<volatile uint8_t *>(valid + (j & 3))[warp & 3] =
                    (uint8_t)(((there & 0xFFFFu) == 0xFFFFu ? 1 : 0) |
                              ((there >> 16) == 0xFFFFu ? 2 : 0));
            {
                uint8_t *dst = smem + S::K + st * S::TILE + sw;
                Meta m[L::NB];
#pragma unroll
                for (int i = 0; i < L::NB; ++i) m[i] = meta_of(km[i]);
#pragma unroll
                for (int w = 0; w < L::D / 8; ++w) {
                    const int c8 = 4 * (w % L::NJ) + w / L::NJ;       // word t * NJ + j
                    const Meta &q = m[c8 * 8 / L::G];
                    *reinterpret_cast<uint4 *>(dst + (c8 >> 3) * (128 * 128) +
                                               (((c8 & 7) ^ (tid & 7)) << 4)) =
                        dequant8(kw[w], q.s, q.z1024, q.z64);
                }
                fence_proxy_async();
                mbar_arrive(bars + KFULL + st);
            }
            // V
            if (j >= STAGES && !warp_wait(bars + VFREE + st, ph ^ 1)) { ok = false; break; }
            {
                uint8_t *dst = smem + S::V + st * S::TILE + sw;
                Meta m[L::NB];
#pragma unroll
                for (int i = 0; i < L::NB; ++i) m[i] = meta_of(vmeta[i]);
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
                        y = dequant8(vw[w], m[u].s, m[u].z1024, m[u].z64);
                    } else {
                        // low halves are nibbles 0-3, high halves 4-7
                        const Meta &a = m[2 * u], &b = m[2 * u + 1];
                        y = dequant8(vw[w], __lows2half2(a.s, b.s), __lows2half2(a.z1024, b.z1024),
                                     __lows2half2(a.z64, b.z64));
                    }
                    *reinterpret_cast<uint4 *>(dst + u * (128 * 128) +
                                               ((g ^ (tid & 7)) << 4)) = y;
                }
                fence_proxy_async();
                mbar_arrive(bars + VFULL + st);
            }
            if (j + 1 < ntile) there = fetch(j + 1);
        }
        if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
    } else {
        // ---------------- MMA ----------------------------------------------
        regs_down<40>();
        if (warp == 12) {
        asm volatile("bar.sync 1, 288;\n" ::: "memory");
        if (lane == 0) {
            bool ok = true;
            const uint32_t q0 = smem_u32(smem + S::Q), k0 = smem_u32(smem + S::K),
                           v0 = smem_u32(smem + S::V);
            constexpr uint32_t IS = idesc(TM, TN, false), IO = idesc(TM, L::D, true);
            auto scores = [&](int qi, int st) {
#pragma unroll
                for (int k = 0; k < L::D / 16; ++k) {
                    const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
                    mma_ss(tm + qi * 128, sdesc(q0 + qi * S::TILE + off, 16, 1024),
                           sdesc(k0 + st * S::TILE + off, 16, 1024), IS, k > 0);
                }
                tm_commit(bars + SFULL + qi);
            };
            auto values = [&](int qi, int st, bool acc) {
#pragma unroll
                for (int k = 0; k < TN / 16; ++k)
                    mma_ts(tm + 256 + qi * L::D, tm + qi * 128 + k * 8,
                           sdesc(v0 + st * S::TILE + k * 2048, 128 * 128, 1024), IO, acc || k > 0);
                tm_commit(bars + OFULL + qi);
            };
            if (ntile > 0) {
                ok = mbar_wait_bounded(bars + KFULL, 0);
                tm_fence_after();
                if (ok) {
                    for (int qi = 0; qi < qtiles; ++qi) scores(qi, 0);
                    tm_commit(bars + KFREE);
                }
            }
            for (int j = 0; ok && j < ntile; ++j) {
                const int st = j % STAGES, ph = (j / STAGES) & 1;
                const int sn = (j + 1) % STAGES, pn = ((j + 1) / STAGES) & 1;
                ok = mbar_wait_bounded(bars + VFULL + st, ph);
                if (!ok) break;
                for (int qi = 0; qi < qtiles; ++qi) {
                    ok = mbar_wait_bounded(bars + PFULL + qi, j & 1);
                    if (!ok) break;
                    tm_fence_after();
                    values(qi, st, j > 0);
                    if (j + 1 < ntile) {
                        if (qi == 0) {
                            ok = mbar_wait_bounded(bars + KFULL + sn, pn);
                            if (!ok) break;
                            tm_fence_after();
                        }
                        scores(qi, sn);
                    }
                }
                if (!ok) break;
                tm_commit(bars + VFREE + st);
                if (j + 1 < ntile) tm_commit(bars + KFREE + sn);
            }
            if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
            // nothing is in flight when tensor memory is given back
            tm_commit(bars + DRAIN);
            mbar_wait_bounded(bars + DRAIN, 0);
        }
        __syncwarp();
        }
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 12) tm_free(tm, 512);
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
