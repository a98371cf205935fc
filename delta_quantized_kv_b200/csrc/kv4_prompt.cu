// kv4_prompt.cu -- prompt attention over the paged 4-bit cache: ragged chunks
// of causal queries, on the 5th-generation tensor cores.
//
// The rows of one kv head are its G query heads of every token, row r of a
// sequence's chunk being token r / G, head r % G.  A job is 256 of them, two
// query tiles of 128 (the M of one tcgen05.mma), and walks the positions it sees
// in tiles of 128.  One CTA per SM takes an equal run of the batch's position
// tiles; a job that a run cuts leaves partial results, which a second kernel
// joins.  Five warpgroups:
//   0, 1   softmax of query tile 0, 1: one thread a row, 64 positions a step;
//          scores from tensor memory, weights back into it as the A operand of
//          the second product
//   2, 3   dequantisation of K, V: one thread a position; packed records from
//          global memory, fp16 values (exact) into swizzled shared memory, two
//          stages each
//   4      a warp for each query tile issues its MMAs
// Tensor memory: scores S0, S1 (fp32 128 x 128 each: two halves of 64
// positions, so that the next step's are computed while the softmax works on
// this one's; the fp16 weights stand over their half) and outputs O0, O1.
//
// A V word holds 8 channels 8 apart, so dequantised words are stored as they
// come: the columns of O are a permutation of the channels, undone in
// registers when O is written.
//
// Softmax, per row: the weights are 2^(x - ref) with ref at least max - 15 and
// at most max - 7 (log2 units); O is rescaled only when the maximum has risen
// by more than 8 since ref was set, so it seldom is.  Weights in [.., 2^15]
// are rounded to fp16 once; sums and scores are fp32.
//
// Measured on one B200: a prompt of 8192 tokens (32 heads over 8, D 128, bf16) in
// 653-660 us a call, 830-840 TFLOP/s (calls queued behind one another: 610-622);
// chunks of 500 and 160 tokens behind 24577 and 13187 positions in 278-281 us,
// 850-860 TFLOP/s (259-262).  A CTA takes 4100-4500 clocks for two query tiles and 128 positions;
// the softmax warps are at work for 90 % of them, the tensor cores for 44 %; ALU
// and exponentials are at 45 %, the issue slots at 55 %.
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
constexpr int SN = 64;             // and per step of the softmax: half a tile
constexpr int THREADS = 640;
constexpr int STAGES = 2;

struct Prompt {
    Query q;
    int G, ctas, slot;             // slot: rows of a partial result
    float *ws;                     // [ctas][2][slot][D + 4] partial rows, then a Part per CTA
    int64_t ws_floats;
};

// A job whose positions several CTAs share: the CTA with its first one leaves
// this, the join kernel adds the shares up.
struct Part {
    int ctas;                      // that share it, this and the following; 0: none
    int kvh, tok0, row0, nrow;
    int pad[3];
};
__device__ inline Part *part_of(const Prompt &p, int D, int cta) {
    return reinterpret_cast<Part *>(p.ws + (int64_t)p.ctas * 2 * p.slot * (D + 4)) + cta;
}
// Row r of a CTA's partial results: kind 0 of the job that it found begun,
// kind 1 of the one that it left unfinished.
__device__ inline float *part_row(const Prompt &p, int D, int cta, int kind, int r) {
    return p.ws + (((int64_t)cta * 2 + kind) * p.slot + r) * (D + 4);
}

template <int D>
struct Smem {
    static constexpr int SLABS = D / 64;            // 64-channel slabs of 128-byte rows
    static constexpr int TILE = SLABS * 128 * 128;  // bytes of a 128-row fp16 tile
    static constexpr int Q = 0;
    static constexpr int K = 2 * TILE;
    static constexpr int V = K + STAGES * TILE;
    static constexpr int BAR = V + STAGES * TILE;
    static constexpr int WALK = BAR + 224 + 64;     // a job list's state per warp
    static constexpr int END = WALK + 20 * 80;
    // one CTA per SM: it takes all of the tensor memory
    static constexpr int BYTES = (END > 120 * 1024 ? END : 120 * 1024) + 1024;
};

// barriers, in 8-byte slots; SFULL, PFULL and OFULL by query tile and half (a
// warp is never two uses of a barrier behind)
enum { KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SFULL = 8, PFULL = 12, OFULL = 16, QFULL = 20,
       DRAIN = 22, N_BAR = 23 };

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
// The same with 16.
__device__ inline void tm_ld16(uint32_t *r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ inline void tm_wait_ld16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" : DKV_RW8(r, 0), DKV_RW8(r, 8)::"memory");
}
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

// Registers of this warpgroup.  640 threads are launched with 96 each; 2 x 144
// + 2 x 72 + 48 = 5 x 96.
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
// Exponent e with max |q| 2^e in [2^14, 2^15).
__device__ inline int q_exponent(float mx) {
    if (!(mx > 0.f)) return 0;
    const int e = 14 - (int)((__float_as_uint(mx) >> 23) & 255u) + 127;
    return max(-100, min(120, e));
}

// ---------------------------------------------------------------------------
// Distribution of the work.  A job is 256 rows of one kv head of one sequence;
// jobs stand in order of sequence, kv head and row.  A job counts the positions
// it sees, times G, and COST position tiles more, as units: they grow by 256
// from block to block until a window fills, so their sums are closed formulas.
// The units of the batch are cut into equal runs, one per CTA: a run may begin
// and end inside a job, and has its position tiles from and up to there.
// ---------------------------------------------------------------------------
// us with 1, 2, 3, 4, 5 (calls queued): a prompt of 8192 708, 657, 615, 604, 609; 24
// short windowed prompts 79.7, 80.0, 82.1, 83.1, 83.9; a chunk behind a long prefix the
// same with all
constexpr int COST = 3;
constexpr int MIN_TILES = 6;       // of a run, where there are enough

struct Seq {
    int n, len, s0, blocks;        // rows' tokens, length, first row, blocks of 256 rows
};
__device__ inline Seq load_seq(const View &v, const Prompt &p, int b) {
    Seq s{0, 0, 0, 0};
    if (b >= v.B) return s;
    s.s0 = seq_start(v, b);
    s.n = (v.starts ? v.starts[b + 1] : s.s0 + v.n_uniform) - s.s0;
    if (s.n <= 0 || s.s0 < 0) return s;
    s.len = seq_len(v, b);
    if (s.len < 0) return s;
    if (s.n > s.len || s.s0 + s.n > v.n_rows) {      // more rows than positions or queries
        set_status(v.status, DKV_DEV_BAD_SEQLEN);
        return s;
    }
    s.blocks = (int)(((int64_t)s.n * p.G + 2 * TM - 1) / (2 * TM));
    return s;
}
// Position tiles that block `blk` sees, and the first one's position.
__device__ inline int tiles_of(const Prompt &p, const Seq &s, int blk, int *kv0) {
    const int row0 = blk * 2 * TM, nrow = s.n * p.G, pos0 = s.len - s.n;
    const int first = pos0 + row0 / p.G, last = pos0 + (min(row0 + 2 * TM, nrow) - 1) / p.G;
    const int lo = p.q.window > 0 ? max(0, first - p.q.window + 1) & ~(RT - 1) : 0;
    *kv0 = lo;
    return (last + 1 - lo + TN - 1) / TN;
}
// Units of blocks 0 .. m - 1, and of block m.
struct Units {
    int64_t base, full;            // block i: base + 256 (i + 1), at most full
    int64_t cost;
};
__device__ inline Units units_of(const Prompt &p, const Seq &s) {
    Units u;
    u.base = (int64_t)p.G * (s.len - s.n);
    u.full = p.q.window > 0 ? (int64_t)p.G * p.q.window + 2 * TM : INT64_MAX;
    u.cost = (int64_t)COST * TN * p.G;
    return u;
}
__device__ inline int64_t units_before(const Units &u, int64_t m) {
    const int64_t k = u.full <= u.base ? 0 : min(m, (u.full - u.base) / (2 * TM));
    return u.base * k + TM * k * (k + 1) + (m > k ? (m - k) * u.full : 0) + m * u.cost;
}
__device__ inline int64_t units_at(const Units &u, int64_t m) {
    return min(u.full, u.base + 2 * TM * (m + 1)) + u.cost;
}
__device__ inline int64_t ctas_used(int64_t total, int G, int ctas) {
    const int64_t least = (int64_t)MIN_TILES * TN * G, n = total / least;
    return n < 1 ? (total > 0) : n < ctas ? n : ctas;
}
// first unit of CTA c, and the CTA of unit u
__device__ inline int64_t unit_of(int64_t c, int64_t total, int64_t n) {
    const int64_t q = total / n, r = total - q * n;
    return c * q + (c < r ? c : r);
}
__device__ inline int64_t cta_of(int64_t u, int64_t total, int64_t n) {
    const int64_t q = total / n, r = total - q * n;
    return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
}

// A CTA's run: where it begins, and its units.
struct Run {
    int b, kvh, blk;
    int64_t off, left;             // units of the first job that others did; units of the run
    int64_t begin, total, n;       // the run's first unit; units and CTAs of the batch
};
__device__ inline Run find_run(const View &v, const Prompt &p, int cta) {
    const int lane = threadIdx.x & 31;
    Run r{};
    auto of_head = [&](int b) {                     // units of one kv head
        const Seq s = load_seq(v, p, b);
        return s.blocks > 0 ? units_before(units_of(p, s), s.blocks) : 0;
    };
    for (int b = lane; b < v.B; b += 32) r.total += of_head(b);
#pragma unroll
    for (int o = 16; o; o >>= 1) r.total += __shfl_xor_sync(0xffffffffu, r.total, o);
    r.total *= v.H;
    r.n = ctas_used(r.total, p.G, p.ctas);
    if (cta >= r.n) return r;                       // left = 0
    r.begin = unit_of(cta, r.total, r.n);
    r.left = unit_of(cta + 1, r.total, r.n) - r.begin;
    int64_t at = r.begin;
    for (int b0 = 0; b0 < v.B; b0 += 32) {
        const int64_t u = b0 + lane < v.B ? of_head(b0 + lane) : 0;
        int64_t inc = u * v.H;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int64_t one = __shfl_sync(0xffffffffu, u, l);
            at -= __shfl_sync(0xffffffffu, inc, l) - one * v.H;
            r.b = b0 + l;
            r.kvh = (int)(at / one);
            at -= r.kvh * one;
            const Seq s = load_seq(v, p, r.b);
            const Units q = units_of(p, s);
            int lo = 0, hi = s.blocks;              // the last block that begins at or before `at`
            while (hi - lo > 1) {
                const int mid = lo + (hi - lo) / 2;
                if (units_before(q, mid) <= at) lo = mid;
                else hi = mid;
            }
            r.blk = lo;
            r.off = at - units_before(q, lo);
            return r;
        }
        at -= __shfl_sync(0xffffffffu, inc, 31);
    }
    r.left = 0;                                     // not reached
    return r;
}

// A job, or the CTA's share of it.
struct Job {
    int b, kvh;
    int row0, nrow;        // first row of the 256, rows of the sequence's chunk (tokens * G)
    int tok0;              // first token row of the sequence in Q
    int pos0;              // position of the chunk's first token
    int len;
    int kv0, ntile;        // first position of the share, position tiles
    bool begins, ends;     // it has the job's first, last tile
    int64_t end;           // unit behind the job
};
// A run's jobs, one after another.  The state stands in shared memory, one for
// each warp: registers are dear, and it is looked at once a job.
struct Walk {
    Run r;
    Seq s;
};
__device__ inline void walk_begin(const View &v, const Prompt &p, const Run &run, Walk *w) {
    const Seq s = run.left > 0 ? load_seq(v, p, run.b) : Seq{0, 0, 0, 0};
    if ((threadIdx.x & 31) == 0) {
        w->r = run;
        w->s = s;
    }
    __syncwarp();
}
__device__ inline bool walk_next(const View &v, const Prompt &p, Walk *w, Job *j) {
    Run r = w->r;
    Seq s = w->s;
    bool got = false;
    __syncwarp();
    while (!got && r.left > 0) {
        int kv0;
        const int tiles = tiles_of(p, s, r.blk, &kv0);
        const Units u = units_of(p, s);
        const int64_t units = units_at(u, r.blk);
        const int64_t rest = units - r.off, take = rest < r.left ? rest : r.left;
        // tiles up to a unit of the job; behind the cost, `each` units a tile (at most
        // 128 G + 257, less than the least run, so that every run inside a job has one)
        const int64_t each = (units - u.cost + tiles - 1) / tiles;
        auto upto = [&](int64_t x) {
            return x <= u.cost ? 0 : x >= units ? tiles : (int)min((int64_t)tiles, (x - u.cost) / each);
        };
        const int t0 = upto(r.off), t1 = upto(r.off + take);
        j->b = r.b;
        j->kvh = r.kvh;
        j->row0 = r.blk * 2 * TM;
        j->nrow = s.n * p.G;
        j->tok0 = s.s0;
        j->pos0 = s.len - s.n;
        j->len = s.len;
        j->kv0 = kv0 + t0 * TN;
        j->ntile = t1 - t0;
        j->begins = t0 == 0;
        j->ends = t1 == tiles;
        j->end = r.begin + rest;
        got = t1 > t0;
        r.begin += take;
        r.left -= take;
        r.off += take;
        if (r.off == units) {
            r.off = 0;
            if (++r.blk == s.blocks) {
                r.blk = 0;
                if (++r.kvh == v.H) {
                    r.kvh = 0;
                    while (r.left > 0) {
                        if (++r.b >= v.B) r.left = 0;
                        s = load_seq(v, p, r.b);
                        if (s.blocks > 0) break;
                    }
                }
            }
        }
    }
    if ((threadIdx.x & 31) == 0) {
        w->r = r;
        w->s = s;
    }
    __syncwarp();
    return got;
}
// Query tiles of a job.
__device__ inline int query_tiles(const Job &j) { return j.nrow - j.row0 > TM ? 2 : 1; }

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

// A block's scale, and its zero point as dequant8 takes it.
struct Meta {
    __half2 s, z1024, z64;
};
__device__ inline Meta meta_of2(uint32_t mm) {     // two blocks: one in each half
    Meta r;
    r.s = meta_scale(mm);
    r.z1024 = u32_as_h2(and_or<0x000F000Fu>(mm, 0x64006400u));
    r.z64 = u32_as_h2(((mm << 4) & 0x00F000F0u) | 0x54005400u);
    return r;
}
__device__ inline Meta meta_of(uint32_t mm, int i) {       // one of them in both
    return meta_of2(prmt(mm, mm, i ? 0x3232u : 0x1010u));
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

// 32 of a row's scores to weights 2^(c s + r), as fp16 and into the sums la, lb.
__device__ inline void weights(const uint32_t (&s)[32], uint64_t c2, uint64_t r2, uint32_t *w,
                               uint64_t &la, uint64_t &lb) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint64_t x = fma2((uint64_t)s[2 * k + 1] << 32 | s[2 * k], c2, r2);
        const uint64_t y = f2(ex2(f2_lo(x)), ex2(f2_hi(x)));
        if (k & 1) lb = add2(lb, y);
        else la = add2(la, y);
        w[k] = pack_h2(f2_lo(y), f2_hi(y));
    }
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
    // dequantising warp).  Tile j + 4's is written once tile j + 2's scores have
    // been computed, which follow the use of tile j's weights.
    volatile uint32_t *valid = tm_slot + 1;
    Run *run = reinterpret_cast<Run *>(smem + S::BAR + 224);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    const int tid = threadIdx.x & 127;
    Walk *walk = reinterpret_cast<Walk *>(smem + S::WALK) + warp;
    static_assert(sizeof(Run) <= 64 && sizeof(Walk) <= 80, "their places in shared memory");

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + KFULL + i, 4);
            mbar_init(bars + KFREE + i, 2);
            mbar_init(bars + VFULL + i, 4);
            mbar_init(bars + VFREE + i, 2);
            mbar_init(bars + QFULL + i, 4);
            for (int k = 0; k < 2; ++k) {
                mbar_init(bars + SFULL + 2 * i + k, 1);
                mbar_init(bars + PFULL + 2 * i + k, 4);
                mbar_init(bars + OFULL + 2 * i + k, 1);
            }
        }
        mbar_init(bars + DRAIN, 2);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 0) {
        if (blockIdx.x == 0) check_starts(v);
        const Run r = find_run(v, p, blockIdx.x);
        if (lane == 0) {
            *run = r;
            Part *x = part_of(p, L::D, blockIdx.x);
            if (range_ok(v.status, x, sizeof(Part), p.ws, p.ws_floats * 4)) x->ctas = 0;
        }
    }
    if (warp == 16) tm_alloc(smem_u32(tm_slot), 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tm = *tm_slot;
    Job job;
    bool ok = true;

    if (wg < 2) {
        // ---------------- softmax ------------------------------------------
        regs_up<144>();
        const int qi = wg;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
        const uint32_t tSP = tm + lane_base + qi * 128, tO = tm + lane_base + 256 + qi * L::D;
        walk_begin(v, p, *run, walk);
        uint32_t step0 = 0, tile0 = 0;     // steps of this warp, tiles of the CTA so far
        while (ok && walk_next(v, p, walk, &job)) {
            if (job.begins && !job.ends && threadIdx.x == 0) {
                Part *x = part_of(p, L::D, blockIdx.x);
                if (range_ok(v.status, x, sizeof(Part), p.ws, p.ws_floats * 4)) {
                    x->kvh = job.kvh;
                    x->tok0 = job.tok0;
                    x->row0 = job.row0;
                    x->nrow = job.nrow;
                    x->ctas = (int)cta_of(job.end - 1, run->total, run->n) - (int)blockIdx.x + 1;
                }
            }
            if (qi >= query_tiles(job)) {
                tile0 += job.ntile;
                continue;
            }
            const int row = job.row0 + qi * TM + tid;
            const bool have = row < job.nrow;
            const int tok = have ? row / p.G : 0;
            const int head = job.kvh * p.G + (have ? row - tok * p.G : 0);
            const int pos = have ? job.pos0 + tok : -1;
            const int lo = p.q.window > 0 ? pos - p.q.window : -1;        // sees (lo, pos]
            float c1 = p.q.scale * 1.44269504088896340736f;
            {
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
                // not 0: hidden scores are -inf, and 0 times that is NaN
                c1 = fmaxf(c1, 1.17549435e-38f);
#pragma unroll
                for (int i = 0; i < L::D / 8; ++i)
                    *reinterpret_cast<uint4 *>(qrow + (i >> 3) * (128 * 128) +
                                               (((i & 7) ^ (tid & 7)) << 4)) = u[i];
                fence_proxy_async();
                warp_arrive(bars + QFULL + qi);
            }
            float neg = 0.f, top = -INFINITY;  // minus the reference; what scores may reach with it
            uint64_t l2 = 0;                   // the sum, in two halves
            const int row_first = job.row0 + qi * TM;
            const int pmin = job.pos0 + row_first / p.G;     // the tile's first and last positions
            const int pmax = job.pos0 + (min(row_first + TM, job.nrow) - 1) / p.G;
            for (int j = 0; j < 2 * job.ntile; ++j) {
                const int h = j & 1;
                const uint32_t at = step0 + j, tS = tSP + h * SN;
                ok = warp_wait(bars + SFULL + 2 * qi + h, (at >> 1) & 1);
                if (!ok) break;
                tm_fence_after();
                const int kv = job.kv0 + j * SN;
                const uint32_t vm = valid[(tile0 + (j >> 1)) & 3] >> (16 * h) & 0x0303u;
                const bool edge = kv + SN - 1 > pmin ||
                                  (p.q.window > 0 && kv <= pmax - p.q.window) || vm != 0x0303u;
                uint32_t w[SN / 2];
                uint64_t la, lb;
                // A job's first step takes its reference from the maximum.  Behind it the
                // weights are taken with the reference as it stands, and the scores'
                // maximum alongside; where it has risen too far (seldom) the step is
                // done again.
                while (true) {
                    uint32_t s0[32], s1[32];
                    tm_ld32(s0, tS);
                    tm_ld32(s1, tS + 32);
                    tm_wait_ld32(s0);
                    tm_wait_ld32(s1);
                    if (edge) {
                        // the row sees (lo, pos], and records that are there
                        auto see = [&](int i) {
                            const int x = kv + 32 * i;
                            const uint32_t v2 = vm >> (8 * i);
                            return below(pos + 1 - x) & ~below(lo + 1 - x) &
                                   ((v2 & 1 ? 0xFFFFu : 0u) | (v2 & 2 ? 0xFFFF0000u : 0u));
                        };
                        hide(s0, see(0));
                        hide(s1, see(1));
                    }
                    const float mx = fmaxf(max32(s0), max32(s1)) * c1;
                    if (j == 0 && mx > -INFINITY) {
                        neg = 7.f - mx;
                        top = mx + 8.f;
                    }
                    const uint64_t c2 = f2(c1, c1), r2 = f2(neg, neg);
                    la = lb = 0;
                    weights(s0, c2, r2, w, la, lb);
                    weights(s1, c2, r2, w + 16, la, lb);
                    // (NaN scores leave mx to the others; their weights are NaN)
                    const bool up = mx > top;
                    if (!__any_sync(0xffffffffu, up)) break;
                    const float f = top == -INFINITY ? 0.f : ex2(7.f - neg - mx);
                    // O must be at rest
                    ok = warp_wait(bars + OFULL + 2 * qi + (h ^ 1), (at - 1) >> 1 & 1);
                    if (!ok) break;
                    tm_fence_after();
#pragma unroll
                    for (int i = 0; i < L::D / 16; ++i) {
                        uint32_t o[16];
                        tm_ld16(o, tO + 16 * i);
                        tm_wait_ld16(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(up ? __uint_as_float(o[k]) * f
                                                      : __uint_as_float(o[k]));
                        tm_st16(tO + 16 * i, o);
                    }
                    if (up) {
                        l2 = fma2(l2, f2(f, f), 0);
                        neg = 7.f - mx;
                        top = mx + 8.f;
                    }
                }
                if (!ok) break;
                l2 = add2(l2, add2(la, lb));
                tm_st32(tS, w);
                tm_wait_st();
                tm_fence_before();
                warp_arrive(bars + PFULL + 2 * qi + h);
            }
            step0 += 2 * job.ntile;
            tile0 += job.ntile;
            // ---------------- output ---------------------------------------
            ok = ok && warp_wait(bars + OFULL + 2 * qi + 1, ((step0 >> 1) - 1) & 1);
            if (!ok) break;
            tm_fence_after();
            const float l = f2_lo(l2) + f2_hi(l2);
            const int64_t orow = (int64_t)(job.tok0 + tok) * p.q.Hq + head;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);       // NaN stays NaN
            float *part = job.begins && job.ends
                              ? nullptr
                              : part_row(p, L::D, blockIdx.x, job.begins, qi * TM + tid);
#pragma unroll
            for (int u = 0; u < L::D / 64; ++u) {
                uint32_t o[64];
                tm_ld32(o, tO + 64 * u);
                tm_ld32(o + 32, tO + 64 * u + 32);
                tm_wait_ld32(o);
                tm_wait_ld32(o + 32);
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
                        part[L::D] = top == -INFINITY ? -INFINITY : -neg;
                        part[L::D + 1] = l;
                    }
                } else if (p.q.lse) {
                    p.q.lse[orow] = l == 0.f ? -INFINITY : (log2f(l) - neg) * 0.69314718055994530942f;
                }
            }
            tm_fence_before();         // O has been read before the next job's weights arrive
        }
        if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
    } else if (wg < 4) {
        // ---------------- dequantisation: K (2), V (3) ---------------------
        regs_down<72>();
        const bool isk = wg == 2;
        uint64_t *full = bars + (isk ? KFULL : VFULL), *free_ = bars + (isk ? KFREE : VFREE);
        constexpr int NM = (L::NB + 1) / 2;         // meta words: two blocks each
        uint4 code[L::D / 32];                      // the words of the tile at hand
        uint32_t meta[NM];
        const int t = tid & (RT - 1);              // the token in its record
        const int code_at = isk ? L::k_word(t, 0) : L::OFF_V + t * L::ROW;
        const int ps = v.page_size, dp = TN / ps, doff = TN - dp * ps;
        // The thread's position in the tile after, its page and offset there; the
        // page's number is loaded a tile ahead of the records.
        const int32_t *pages = nullptr;
        int at = 0, pi = 0, off = 0, page = 0, left = 0;
        walk_begin(v, p, *run, walk);
        auto open = [&]() {                         // the next job
            left = 0;
            if (!walk_next(v, p, walk, &job)) return;
            left = job.ntile;
            pages = v.table + (int64_t)job.b * v.max_pages;
            at = job.kv0 + tid;
            pi = at / ps;
            off = at - pi * ps;
            page = at < job.len ? pages[pi] : 0;
        };
        // The record of the position, and whether it is as it should be: one that
        // is missing below the length (a bad page) is not seen.
        auto locate = [&](bool *fine) {
            const uint8_t *rec = nullptr;
            *fine = at >= job.len;
            if (!*fine) {
                if (page < 0 || page >= v.n_pages) {
                    set_status(v.status, DKV_DEV_BAD_PAGE);
                } else {
                    rec = v.pool + page * v.page_bytes +
                          ((int64_t)job.kvh * v.rpp + off / RT) * L::REC;
                    if (!range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes))
                        rec = nullptr;
                }
                *fine = rec != nullptr;
            }
            if (--left > 0) {
                at += TN;
                pi += dp;
                off += doff;
                if (off >= ps) {
                    off -= ps;
                    ++pi;
                }
                page = at < job.len ? pages[pi] : 0;
            } else {
                open();
            }
            return rec;
        };
        auto load = [&](const uint8_t *rec, int i) {
            code[i] = rec ? reinterpret_cast<const uint4 *>(rec + code_at)[i] : make_uint4(0, 0, 0, 0);
        };
        auto load_meta = [&](const uint8_t *rec) {
#pragma unroll
            for (int i = 0; i < NM; ++i) meta[i] = 0u;
            if (rec) {
#pragma unroll
                for (int i = 0; i < L::NB; ++i)
                    meta[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(
                                       rec + (isk ? L::k_meta(t, i) : L::v_meta(t, i)))
                                   << (16 * (i & 1));
            }
        };
        open();
        bool more = left > 0, here = true;
        if (more) {
            const uint8_t *rec = locate(&here);
#pragma unroll
            for (int i = 0; i < L::D / 32; ++i) load(rec, i);
            load_meta(rec);
        }
        for (uint32_t j = 0; more; ++j) {
            const int st = j % STAGES, ph = (j / STAGES) & 1;
            const unsigned there = __ballot_sync(0xffffffffu, here);
            more = left > 0;
            const uint8_t *rec = more ? locate(&here) : nullptr;      // the tile after
            if (j >= STAGES && !warp_wait(free_ + st, ph ^ 1)) { ok = false; break; }
            uint8_t *dst = smem + (isk ? S::K : S::V) + st * S::TILE + tid * 128;
            // four words at a time
            if (isk) {
                if (lane == 0)          // two records a warp: lanes 0..15 and 16..31
                    reinterpret_cast<volatile uint8_t *>(valid + (j & 3))[warp & 3] =
                        (uint8_t)(((there & 0xFFFFu) == 0xFFFFu ? 1 : 0) |
                                  ((there >> 16) == 0xFFFFu ? 2 : 0));
                Meta m[L::NB];
#pragma unroll
                for (int i = 0; i < L::NB; ++i) m[i] = meta_of(meta[i / 2], i & 1);
#pragma unroll
                for (int i = 0; i < L::D / 32; ++i) {
                    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                    uint4 y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c8 = 4 * (k % L::NJ) + (4 * i + k) / L::NJ;   // word c8's 8 channels
                        const Meta &q = m[c8 * 8 / L::G];
                        y[k] = dequant8(w[k], q.s, q.z1024, q.z64);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c8 = 4 * (k % L::NJ) + (4 * i + k) / L::NJ;
                        *reinterpret_cast<uint4 *>(dst + (c8 >> 3) * (128 * 128) +
                                                   (((c8 & 7) ^ (tid & 7)) << 4)) = y[k];
                    }
                }
            } else {
                const int flip = L::D == 128 ? ((t >> 1) & 1) << 2 : 0;
                // a word's nibbles are channels 64 u + 16 (n / 2) + 8 (n % 2) + g of
                // chunk g: two blocks of 32 channels (nibbles 0-3: low halves of the
                // pairs, and 4-7: high halves), or one of 64
                Meta m[L::D / 64];
#pragma unroll
                for (int u = 0; u < L::D / 64; ++u)
                    m[u] = L::G == 64 ? meta_of(meta[u / 2], u & 1) : meta_of2(meta[u % NM]);
#pragma unroll
                for (int i = 0; i < L::D / 32; ++i) {
                    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                    uint4 y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const Meta &q = m[L::D == 128 ? k & 1 : 0];
                        y[k] = dequant8(w[k], q.s, q.z1024, q.z64);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // D = 128: words 2 c + u of chunk c ^ flip
                        const int u = L::D == 128 ? k & 1 : 0;
                        const int g = (L::D == 128 ? 2 * i + (k >> 1) : 4 * i + k) ^ flip;
                        *reinterpret_cast<uint4 *>(dst + u * (128 * 128) + ((g ^ (tid & 7)) << 4)) = y[k];
                    }
                }
            }
            fence_proxy_async();
            warp_arrive(full + st);
            // the next tile's words, behind the fence: it waits for loads too
#pragma unroll
            for (int i = 0; i < L::D / 32; ++i) load(rec, i);
            load_meta(rec);
        }
        if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
    } else {
        // ---------------- MMA ----------------------------------------------
        // A warp for each query tile: while one waits, the tensor cores work for
        // the other.  The warp walks in step, one thread of it issues: everything
        // the instructions take is the same in all lanes.
        regs_down<48>();
        const int qi = __shfl_sync(0xffffffffu, warp, 0) - 16;
        if (qi < 2) {
            constexpr uint32_t IS = idesc(TM, SN, false), IO = idesc(TM, L::D, true);
            constexpr uint32_t HI = desc_hi(1024);
            const bool leader = elect_one();
            const uint32_t tS = __shfl_sync(0xffffffffu, tm, 0) + qi * 128,
                           tO = __shfl_sync(0xffffffffu, tm, 0) + 256 + qi * L::D;
            const uint32_t q0 = desc_lo(smem_u32(smem + S::Q + qi * S::TILE), 16),
                           k0 = desc_lo(smem_u32(smem + S::K), 16),
                           v0 = desc_lo(smem_u32(smem + S::V), 128 * 128);
            // half h of position tile i (of the CTA's)
            auto scores = [&](uint32_t i, int h) {
                const uint32_t b = k0 + i % STAGES * (S::TILE >> 4) + h * (SN * 128 >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < L::D / 16; ++k) {
                        const uint32_t off = (k >> 2) * (128 * 128 >> 4) + (k & 3) * (32 >> 4);
                        mma_ss<HI, HI, IS>(tS + h * SN, q0 + off, b + off, k > 0);
                    }
                    tm_commit(bars + SFULL + 2 * qi + h);
                    if (h) tm_commit(bars + KFREE + i % STAGES);
                }
                __syncwarp();
            };
            auto values = [&](uint32_t i, int h, bool acc) {
                const uint32_t b = v0 + i % STAGES * (S::TILE >> 4) + h * (SN * 128 >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < SN / 16; ++k)
                        mma_ts<HI, IO>(tO, tS + h * SN + k * 8, b + k * (2048 >> 4), acc || k > 0);
                    tm_commit(bars + OFULL + 2 * qi + h);
                    if (h) tm_commit(bars + VFREE + i % STAGES);
                }
                __syncwarp();
            };
            walk_begin(v, p, *run, walk);
            uint32_t i0 = 0, q_phase = 0, p_phase = 0;     // tiles of the CTA, jobs and tiles of this warp
            while (ok && walk_next(v, p, walk, &job)) {
                if (qi >= query_tiles(job)) {
                    // nothing to multiply: only its word that the tiles may go
                    for (int i = 0; ok && i < job.ntile; ++i, ++i0) {
                        ok = warp_wait(bars + KFULL + i0 % STAGES, (i0 / STAGES) & 1);
                        if (lane == 0) mbar_arrive(bars + KFREE + i0 % STAGES);
                        ok = ok && warp_wait(bars + VFULL + i0 % STAGES, (i0 / STAGES) & 1);
                        if (lane == 0) mbar_arrive(bars + VFREE + i0 % STAGES);
                    }
                    continue;
                }
                ok = warp_wait(bars + QFULL + qi, q_phase) &&
                     warp_wait(bars + KFULL + i0 % STAGES, (i0 / STAGES) & 1);
                q_phase ^= 1;
                if (!ok) break;
                tm_fence_after();
                scores(i0, 0);
                scores(i0, 1);
                // The scores are taken two steps ahead, into the half of S that the
                // values' product has just read the weights from.
                for (int i = 0; ok && i < job.ntile; ++i, ++i0) {
                    const bool more = i + 1 < job.ntile;
                    const uint32_t n = i0 + 1;
                    ok = warp_wait(bars + VFULL + i0 % STAGES, (i0 / STAGES) & 1);
                    if (more) ok = ok && warp_wait(bars + KFULL + n % STAGES, (n / STAGES) & 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && warp_wait(bars + PFULL + 2 * qi + h, p_phase);
                        if (!ok) break;
                        tm_fence_after();
                        values(i0, h, i > 0 || h > 0);
                        if (more) scores(n, h);
                    }
                    p_phase ^= 1;
                }
            }
            if (!ok) set_status(v.status, DKV_DEV_TIMEOUT);
            // nothing is in flight when tensor memory is given back
            if (leader) tm_commit(bars + DRAIN);
            __syncwarp();
            warp_wait(bars + DRAIN, 0);
        }
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 16) tm_free(tm, 512);
}

// Joins the shares of a job that several CTAs had: block (CTA that began it,
// 8 rows), a warp a row.
template <int D, int DT>
__global__ void __launch_bounds__(256)
join_kernel(View v, Prompt p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const Part *x = part_of(p, D, blockIdx.x);
    if (!range_ok(v.status, x, sizeof(Part), p.ws, p.ws_floats * 4)) return;
    const int n = x->ctas, row = x->row0 + r;
    if (n == 0 || r >= p.slot || row >= x->nrow) return;
    const int tok = row / p.G;
    const int64_t orow = (int64_t)(x->tok0 + tok) * p.q.Hq + x->kvh * p.G + row - tok * p.G;
    constexpr int W = D / 32;
    float m = -INFINITY, l = 0.f, o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = 0.f;
    for (int s = 0; s < n; ++s) {
        const float *y = part_row(p, D, blockIdx.x + s, s == 0, r);
        if (!range_ok(v.status, y, (D + 4) * 4, p.ws, p.ws_floats * 4)) return;
        const float ms = y[D], ls = y[D + 1];
        const float mx = fmaxf(m, ms), ref = mx == -INFINITY ? 0.f : mx;
        const float f0 = ex2(m - ref), f1 = ex2(ms - ref) * ls;     // the parts are normalised
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = fmaf(o[i], f0, y[lane * W + i] * f1);
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
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.q.out) + orow * D) +
                    lane * (W / 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) dst[i] = w[i];
    if (p.q.lse && lane == 0)
        p.q.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
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

// The grid: one CTA per SM, fewer where the call cannot have MIN_TILES for each;
// rows of a partial result.
struct Grid {
    int ctas, slot;
};
cudaError_t grid_of(const View &v, int Hq, Grid *g) {
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)v.n_rows * (Hq / v.H);
    // every sequence may end inside a block
    const int64_t jobs = (rows / (2 * TM) + (v.B < v.n_rows ? v.B : v.n_rows)) * v.H;
    const int64_t tiles = (int64_t)v.max_pages * v.page_size / TN + 2;
    const int64_t ctas = (jobs * (tiles + COST) + MIN_TILES - 1) / MIN_TILES;
    g->ctas = (int)(ctas < sms ? ctas : sms);
    g->slot = (int)(rows < 2 * TM ? rows : 2 * TM);
    return cudaSuccess;
}
int64_t floats_of(const Grid &g, int D) {
    return (int64_t)g.ctas * (2 * g.slot * (D + 4) + sizeof(Part) / 4);
}

template <typename L, int DT>
cudaError_t launch(const View &v, const Prompt &p, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem_once(prompt_kernel<L, DT>, Smem<L::D>::BYTES, &done);
    if (e == cudaSuccess)
        e = launch_pdl(prompt_kernel<L, DT>, dim3(p.ctas), dim3(THREADS), Smem<L::D>::BYTES, st, v,
                       p);
    if (e == cudaSuccess && p.ctas > 1)
        e = launch_pdl(join_kernel<L::D, DT>, dim3(p.ctas, (p.slot + 7) / 8), dim3(256), 0, st, v, p);
    return e;
}
template <typename L>
cudaError_t launch_dt(const View &v, const Prompt &p, cudaStream_t st) {
    return p.q.dtype == DKV_F16 ? launch<L, DKV_F16>(v, p, st) : launch<L, DKV_BF16>(v, p, st);
}

}  // namespace

cudaError_t prompt_workspace_floats(const View &v, int D, int Hq, int64_t *floats) {
    Grid g;
    const cudaError_t e = grid_of(v, Hq, &g);
    if (e != cudaSuccess) return e;
    *floats = floats_of(g, D);
    return cudaSuccess;
}

cudaError_t launch_prompt(const View &v, int D, int G, const Query &q, float *ws,
                          int64_t ws_floats, cudaStream_t st) {
    Grid g;
    const cudaError_t e = grid_of(v, q.Hq, &g);
    if (e != cudaSuccess) return e;
    Prompt p;
    p.q = q;
    p.G = q.Hq / v.H;
    p.ctas = g.ctas;
    p.slot = g.slot;
    p.ws = ws;
    p.ws_floats = ws_floats;
    if (D == 128)
        return G == 32 ? launch_dt<Lay<128, 32>>(v, p, st) : launch_dt<Lay<128, 64>>(v, p, st);
    return G == 32 ? launch_dt<Lay<64, 32>>(v, p, st) : launch_dt<Lay<64, 64>>(v, p, st);
}

}  // namespace kv4
}  // namespace dkv
