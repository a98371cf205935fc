// kv4_decode.cu -- decode attention over the paged 4-bit cache: one to a few
// causal queries per sequence.
//
// The queries of one kv head (nq * G virtual heads) are taken in groups of 8,
// the N of mma.sync m16n8k16; each group streams the sequence's records once.
// A unit is 32 positions (two records) of one (sequence, kv head, head group).
// The units of the batch are flattened and cut into equal runs, one per warp;
// a warp keeps a ring of NST units in flight with bulk copies.  A warp that
// passes the end of a sequence writes a partial (max, sum, output) record; the
// runs still open at the end are combined inside the CTA first, so a
// sequence leaves about one record per CTA that touches it.  The merge kernel
// joins them.
//
// Measured on one B200: 16 sequences of 32768 positions, 64 heads over 8, D 128,
// bf16: 163 us, 3.7 TB/s of packed cache.  Bound by latency: a unit is one chain
// (scores, maximum, vote, exponentials, products), and 3.7 warps a scheduler fill
// 56 % of the issue slots (860 instructions a unit at 8192 positions a sequence),
// the ALU 54 % (masks and shifts of the codes), the tensor cores 19 %, DRAM 44 %.
//
// Mathematics.  x^ = (c - z) s, so with the sum over a block's channels
//   q . k^ = sum_b s_b (q_b . c_b) + sum_b (s_b z_b) (-sum q_b):
// the codes go into the MMA as they are -- a masked nibble IS the fp16
// subnormal c 2^-24 (or c 2^-20), exact, no subtraction -- the blocks'
// partial products are scaled in fp32, and the zero points are one more small
// MMA whose A operand s z is exact in fp16 and whose B operand, the query's
// block sums, is an fp16 hi + lo pair.  For the output,
//   sum_p P_p v^_p = sum_p (P_p s_pb) c_p - sum_p P_p (s_pb z_pb):
// the weights are rounded to fp16 once (P); the product P s is taken as fp16
// hi for bf16 outputs, and as a hi + lo pair (two MMAs) for fp16 ones, whose own
// rounding is 8 times finer: exact for P s from 2^-7 on.
// Ranges: a query is scaled by a power of two so its largest element lies in
// [2^14, 2^15); P is scaled by 2^k with k from the largest V scale that the
// warp's queries have seen so far (P s <= 2^14, k <= 15), as part of the running
// maximum, so rescaling is the online softmax's own.  Small products end in
// fp16's subnormals: with the largest weight as 1, a weight times a scale is off
// by at most 2^-25-k, which is 2^-38 of the largest scale seen, or 2^-40.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "kv4_common.cuh"
#include "kv4_internal.h"

namespace dkv {
namespace kv4 {
namespace {

constexpr int WARPS = 8;          // per CTA
constexpr int CTAS_PER_SM = 2;    // 16 warps: 128 registers each
constexpr int NST = 3;            // units in flight per warp (2: the same times)
constexpr int UT = 2 * RT;        // positions per unit
constexpr int64_t MIN_UNITS = 2;  // per warp (one user's 4096 positions: 13.8 us with 1 or 2, 16.4 with 4)

struct Split {
    Query q;
    int nq, G, nhg, nseq;   // nseq: H * nhg runs of records per batch entry
    float *ws;
    int64_t ws_floats;
    int NW;                 // warps of the grid
    int unsent;             // bytes announced of each unit that no copy brings: 0 but in tests
};

template <int D>
__host__ __device__ constexpr int rec_floats() { return 16 + 8 * D; }   // m[8], l[8], o[8][D]

// First position of sequence length `len` that any of the nq queries sees,
// down to a record's start; units of 32 positions up to len.
__device__ inline int span(int len, int nq, int window, int *first) {
    int lo = 0;
    if (window > 0) lo = max(0, len - nq + 1 - window);
    lo &= ~(RT - 1);
    *first = lo;
    return len > 0 ? (len - lo + UT - 1) / UT : 0;
}

__device__ inline int64_t warps_used(int64_t total, int NW) {
    const int64_t w = (total + MIN_UNITS - 1) / MIN_UNITS;
    return w < 1 ? 1 : (w < NW ? w : NW);
}
// first unit of warp w
__device__ inline int64_t unit_of(int64_t w, int64_t total, int64_t nw) {
    const int64_t q = total / nw, r = total - q * nw;
    return w * q + (w < r ? w : r);
}
// warp that owns unit u
__device__ inline int64_t warp_of(int64_t u, int64_t total, int64_t nw) {
    const int64_t q = total / nw, r = total - q * nw;
    return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
}

// Units of all batch entries, of those before b, and of one run of b; a whole
// warp asking.
__device__ inline void units_around(const View &v, const Split &p, int b, int64_t *total,
                                    int64_t *before, int *own) {
    const int lane = threadIdx.x & 31;
    int64_t n = 0, m = 0;
    int mine = 0;
    for (int i = lane; i < v.B; i += 32) {
        int first;
        const int k = span(max(0, seq_len(v, i)), p.nq, p.q.window, &first);
        n += k;
        if (i < b) m += k;
        if (i == b) mine = k;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    *total = n * p.nseq;
    *before = m * p.nseq;
    *own = __reduce_max_sync(0xffffffffu, mine);
}
// Units of all batch entries.
__device__ inline int64_t units_of_all(const View &v, const Split &p) {
    const int lane = threadIdx.x & 31;
    int64_t n = 0;
    for (int b = lane; b < v.B; b += 32) {
        int first;
        n += span(max(0, seq_len(v, b)), p.nq, p.q.window, &first);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n * p.nseq;
}

// A position in the flattened units.
struct Cursor {
    int b, sq, u;          // batch entry, run (kv head * nhg + head group), unit
    int nu, first, len;    // of this batch entry
};

__device__ inline void load_entry(const View &v, const Split &p, Cursor &c) {
    c.nu = 0;
    while (c.b < v.B) {
        c.len = max(0, seq_len(v, c.b));
        c.nu = span(c.len, p.nq, p.q.window, &c.first);
        if (c.nu > 0) break;
        ++c.b;
    }
}
__device__ inline void step(const View &v, const Split &p, Cursor &c) {
    if (++c.u < c.nu) return;
    c.u = 0;
    if (++c.sq < p.nseq) return;
    c.sq = 0;
    ++c.b;
    load_entry(v, p, c);
}

// The cursor at unit `u0` (< total), a whole warp asking.
__device__ inline Cursor seek(const View &v, const Split &p, int64_t u0) {
    const int lane = threadIdx.x & 31;
    int64_t left = u0;
    Cursor c{};
    for (int b0 = 0; b0 < v.B; b0 += 32) {
        int first, n = 0;
        if (b0 + lane < v.B) n = span(max(0, seq_len(v, b0 + lane)), p.nq, p.q.window, &first);
        int64_t inc = (int64_t)n * p.nseq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int nn = __shfl_sync(0xffffffffu, n, l);
            const int64_t before = __shfl_sync(0xffffffffu, inc, l) - (int64_t)nn * p.nseq;
            c.b = b0 + l;
            left -= before;
            c.sq = (int)(left / nn);
            c.u = (int)(left - (int64_t)c.sq * nn);
            load_entry(v, p, c);
            return c;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
    c.b = v.B;
    return c;
}

__device__ inline void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0));
}
__device__ inline float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// Power of two e with max |q| 2^e in [2^14, 2^15) (0 for a zero row).
__device__ inline int q_exponent(float mx) {
    if (!(mx > 0.f)) return 0;
    const int e = 14 - (int)((__float_as_uint(mx) >> 23) & 255u) + 127;
    return max(-100, min(120, e));
}

// One warp's queries of a head group as MMA B fragments, per lane (g, t):
// column g is virtual head hg * 8 + g.
template <typename L>
struct QFrag {
    uint32_t b[L::D / 16][2];
    uint32_t z;             // the block sums, negated, hi or lo: B of the zero-point MMA
    float c1[2], c2[2];     // score factors of heads 2t, 2t+1 (log2 units)
    int lim[2];             // positions below which heads 2t, 2t+1 see (exclusive)
};

template <typename L, int DT>
__device__ inline void load_q(const View &v, const Split &p, int b, int sq, int len, QFrag<L> &f) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int kvh = sq / p.nhg, hg = sq - kvh * p.nhg;
    const int vh = hg * 8 + g, nv = p.nq * p.G;
    float x[L::NJ * 8];
    float mx = 0.f;
    const int qt = vh / p.G, qh = kvh * p.G + vh - qt * p.G;
    const int64_t base = ((int64_t)b * p.nq + qt) * p.q.tok + (int64_t)qh * p.q.head;
#pragma unroll
    for (int j = 0; j < L::NJ; ++j) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (vh < nv)
            a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q.q) + base +
                                                 32 * j + 8 * t);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (DT == DKV_F16) {
                x[8 * j + 2 * k] = h_lo(w[k]);
                x[8 * j + 2 * k + 1] = h_hi(w[k]);
            } else {
                x[8 * j + 2 * k] = __uint_as_float(w[k] << 16);
                x[8 * j + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
            mx = fmaxf(mx, fmaxf(fabsf(x[8 * j + 2 * k]), fabsf(x[8 * j + 2 * k + 1])));
        }
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = q_exponent(mx);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    float sum[L::NB];
#pragma unroll
    for (int i = 0; i < L::NB; ++i) sum[i] = 0.f;
#pragma unroll
    for (int j = 0; j < L::NJ; ++j) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[8 * j + k] *= up;
            // the sum of what the MMA multiplies (a query element far below the
            // row's largest may lose bits to fp16)
            x[8 * j + k] = __half2float(__float2half_rn(x[8 * j + k]));
            sum[32 * j / L::G] += x[8 * j + k];
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f.b[2 * j + s][0] = pack_h2(x[8 * j + 4 * s], x[8 * j + 4 * s + 1]);
            // these meet the nibbles read as c 2^-20
            f.b[2 * j + s][1] =
                pack_h2(x[8 * j + 4 * s + 2] * 0.0625f, x[8 * j + 4 * s + 3] * 0.0625f);
        }
    }
#pragma unroll
    for (int i = 0; i < L::NB; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        sum[i] *= -0.0009765625f;                       // 2^-10: inside fp16
    }
    // k = 2t, 2t+1 of the k8 MMA: hi of blocks 0..NB-1, then lo
    float hi[2] = {0.f, 0.f}, lo[2] = {0.f, 0.f};
    if (L::NB == 4) {
        hi[0] = (t & 1) ? sum[L::NB - 2] : sum[0];
        hi[1] = (t & 1) ? sum[L::NB - 1] : sum[L::NB > 1 ? 1 : 0];
    } else if (L::NB == 2) {
        hi[0] = sum[0];
        hi[1] = sum[L::NB - 1];
    } else {
        hi[0] = sum[0];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float h = __half2float(__float2half_rn(hi[i]));
        lo[i] = hi[i] - h;
        hi[i] = h;
    }
    const int lo_t = L::NB == 4 ? 2 : 1;                // the lanes that carry the lo parts
    const bool is_lo = t >= lo_t, none = t >= 2 * lo_t;
    f.z = none ? 0u : is_lo ? pack_h2(lo[0], lo[1]) : pack_h2(hi[0], hi[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int h = 2 * t + i;
        const int eh = __shfl_sync(0xffffffffu, e, 4 * h);
        const float down = __uint_as_float((uint32_t)(127 - eh) << 23) * p.q.scale *
                           1.44269504088896340736f;
        f.c1[i] = down * 16777216.f;                    // 2^24
        f.c2[i] = down * 1024.f;
        const int hv = hg * 8 + h;
        f.lim[i] = hv < nv ? len - (p.nq - 1 - hv / p.G) : 0;
    }
}

// Running state of one open sequence.
template <typename L>
struct Acc {
    float o[L::D / 16][4];
    float z[4];
    float m[2], l[2];     // reference (max - k) in log2 units; sum
    int k;                // weights are scaled by 2^k
    uint32_t thr;         // fp16x2 bound of the V scales that k allows
};

template <typename L>
__device__ inline void acc_reset(Acc<L> &a) {
#pragma unroll
    for (int i = 0; i < L::D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a.o[i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) a.z[j] = 0.f;
    a.m[0] = a.m[1] = -INFINITY;
    a.l[0] = a.l[1] = 0.f;
    a.k = 15;
    a.thr = 0x38003800u;   // 0.5
}

// One unit: bit mask of the records that are there, pos of the first's positions;
// edge: some query does not see all 32 of them, and [lo, hi) are those that any sees.
template <typename L, bool LO>
__device__ inline void unit(const uint8_t *st, int mask, int pos, bool edge, int lo, int hi,
                            int window, const QFrag<L> &q, Acc<L> &a) {
    constexpr int NB = L::NB, NJ = L::NJ;
    constexpr uint32_t M0 = 0x000F000Fu, M1 = 0x00F000F0u;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tg = (g >> 1) + 4 * (g & 1);        // token of MMA row g; row g + 8: tg + 8
    float x[2][4];
    uint32_t zm[2][2] = {{0u, 0u}, {0u, 0u}};     // V meta of block g: tokens (t, t+4), (t+8, t+12)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (!(mask >> r & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[r][i] = -INFINITY;
            continue;
        }
        const uint8_t *rec = st + r * L::REC;
        uint32_t wa[NJ], wb[NJ];
        const uint8_t *ra = rec + L::k_slot(tg) * L::ROW + t * NJ * 4;
        const uint8_t *rb = rec + L::k_slot(tg + 8) * L::ROW + t * NJ * 4;
        uint32_t ma[(NB + 1) / 2], mb[(NB + 1) / 2];
        if constexpr (NJ == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(ra);
            const uint4 w = *reinterpret_cast<const uint4 *>(rb);
            wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
            wb[0] = w.x; wb[1] = w.y; wb[2] = w.z; wb[3] = w.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(ra);
            const uint2 w = *reinterpret_cast<const uint2 *>(rb);
            wa[0] = u.x; wa[1] = u.y;
            wb[0] = w.x; wb[1] = w.y;
        }
        const uint8_t *pa = rec + L::k_meta(tg, 0), *pb = rec + L::k_meta(tg + 8, 0);
        if constexpr (NB == 4) {
            const uint2 u = *reinterpret_cast<const uint2 *>(pa);
            const uint2 w = *reinterpret_cast<const uint2 *>(pb);
            ma[0] = u.x; ma[1] = u.y;
            mb[0] = w.x; mb[1] = w.y;
        } else if constexpr (NB == 2) {
            ma[0] = *reinterpret_cast<const uint32_t *>(pa);
            mb[0] = *reinterpret_cast<const uint32_t *>(pb);
        } else {
            ma[0] = *reinterpret_cast<const uint16_t *>(pa);
            mb[0] = *reinterpret_cast<const uint16_t *>(pb);
        }
        if (g < NB) {
            const uint2 u = *reinterpret_cast<const uint2 *>(rec + L::v_meta(t, g));
            zm[r][0] = u.x;
            zm[r][1] = u.y;
        }
        // zero points: (s z) . (-block sums)
        const uint32_t za = (NB == 4 && (t & 1)) ? ma[NB == 4 ? 1 : 0] : ma[0];
        const uint32_t zb = (NB == 4 && (t & 1)) ? mb[NB == 4 ? 1 : 0] : mb[0];
        float zs[4] = {0.f, 0.f, 0.f, 0.f};
        mma1688(zs, h2_as_u32(__hmul2(meta_scale(za), meta_zero(za))),
                h2_as_u32(__hmul2(meta_scale(zb), meta_zero(zb))), q.z);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = b * (NJ / NB); j < (b + 1) * (NJ / NB); ++j) {
                const uint32_t a8 = wa[j] >> 8, b8 = wb[j] >> 8;
                mma16816(d, wa[j] & M0, wb[j] & M0, wa[j] & M1, wb[j] & M1, q.b[2 * j][0],
                         q.b[2 * j][1]);
                mma16816(d, a8 & M0, b8 & M0, a8 & M1, b8 & M1, q.b[2 * j + 1][0],
                         q.b[2 * j + 1][1]);
            }
            const uint32_t ua = ma[b >> 1] & 0xFFF0FFF0u, ub = mb[b >> 1] & 0xFFF0FFF0u;
            const float fa = (b & 1) ? h_hi(ua) : h_lo(ua), fb = (b & 1) ? h_hi(ub) : h_lo(ub);
            s[0] = fmaf(fa, d[0], s[0]);
            s[1] = fmaf(fa, d[1], s[1]);
            s[2] = fmaf(fb, d[2], s[2]);
            s[3] = fmaf(fb, d[3], s[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[r][i] = fmaf(s[i], q.c1[i & 1], zs[i] * q.c2[i & 1]);
        if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = pos + r * RT + tg + (i >> 1) * 8;
                const bool seen = at < q.lim[i & 1] && (window <= 0 || at >= q.lim[i & 1] - window);
                if (!seen) x[r][i] = -INFINITY;
            }
            // nor do leftovers behind the length, or before every window, have a
            // say in the weights' power of two
            auto keep = [&](int at) {
                return (at >= lo && at < hi ? 0xFFFFu : 0u) |
                       (at + 4 >= lo && at + 4 < hi ? 0xFFFF0000u : 0u);
            };
            zm[r][0] &= keep(pos + r * RT + t);
            zm[r][1] &= keep(pos + r * RT + t + 8);
        }
    }
    // the largest V scale bounds the weights' power of two
    constexpr uint32_t ABS = 0x7FFF7FFFu;
    const uint32_t zmax = __vmaxu2(__vmaxu2(zm[0][0] & ABS, zm[0][1] & ABS),
                                   __vmaxu2(zm[1][0] & ABS, zm[1][1] & ABS));
    int k = a.k;
    if (__any_sync(0xffffffffu, __vmaxu2(zmax, a.thr) != a.thr)) {
        unsigned mx = max(zmax & 0xFFFFu, zmax >> 16);
        mx = __reduce_max_sync(0xffffffffu, mx) | 0xFu;
        const int e = (int)(mx >> 10) - 14;           // s < 2^e
        k = min(15, 14 - e);
        const uint32_t b = (uint32_t)(14 - k + 15) << 10;   // 2^(14 - k)
        a.thr = b | b << 16;
    }
    float mn[2] = {fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])),
                   fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]))};
    bool moved = k != a.k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 4));
        mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 8));
        mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 16));
        mn[i] = fmaxf(a.m[i] + (float)a.k, mn[i]) - (float)k;
        moved |= mn[i] > a.m[i];
    }
    a.k = k;
    if (__any_sync(0xffffffffu, moved)) {
        // o's columns are heads 2t, 2t+1, like the scores'
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = mn[i] > a.m[i] ? ex2(a.m[i] - mn[i]) : 1.f;
            a.l[i] *= f;
            a.z[i] *= f;
#pragma unroll
            for (int c = 0; c < L::D / 16; ++c) {
                a.o[c][i] *= f;
                a.o[c][i + 2] *= f;
            }
            a.m[i] = fmaxf(a.m[i], mn[i]);
        }
    }
    const float ref0 = a.m[0] == -INFINITY ? 0.f : a.m[0];
    const float ref1 = a.m[1] == -INFINITY ? 0.f : a.m[1];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (!(mask >> r & 1)) continue;
        const float p0 = ex2(x[r][0] - ref0), p1 = ex2(x[r][1] - ref1);
        const float p2 = ex2(x[r][2] - ref0), p3 = ex2(x[r][3] - ref1);
        a.l[0] += p0 + p2;
        a.l[1] += p1 + p3;
        // B fragments: head g, tokens (t, t+4) and (t+8, t+12)
        const uint32_t b0 = movm_t(pack_h2(p0, p1)), b1 = movm_t(pack_h2(p2, p3));
        const uint8_t *rec = st + r * L::REC;
        mma16816(a.z, h2_as_u32(__hmul2(meta_scale(zm[r][0]), meta_zero(zm[r][0]))), 0u,
                 h2_as_u32(__hmul2(meta_scale(zm[r][1]), meta_zero(zm[r][1]))), 0u, b0, b1);
        uint32_t sm[NB][2];
        if constexpr (NB == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(rec + L::v_meta(t, 0));
            const uint4 w = *reinterpret_cast<const uint4 *>(rec + L::v_meta(t, 2));
            sm[0][0] = u.x; sm[0][1] = u.y; sm[1][0] = u.z; sm[1][1] = u.w;
            sm[2][0] = w.x; sm[2][1] = w.y; sm[3][0] = w.z; sm[3][1] = w.w;
        } else if constexpr (NB == 2) {
            const uint4 u = *reinterpret_cast<const uint4 *>(rec + L::v_meta(t, 0));
            sm[0][0] = u.x; sm[0][1] = u.y; sm[1][0] = u.z; sm[1][1] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(rec + L::v_meta(t, 0));
            sm[0][0] = u.x; sm[0][1] = u.y;
        }
        uint32_t h[NB][2], lo[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const __half2 s0 = meta_scale(sm[b][0]), s1 = meta_scale(sm[b][1]);
            const __half2 h0 = __hmul2(u32_as_h2(b0), s0), h1 = __hmul2(u32_as_h2(b1), s1);
            h[b][0] = h2_as_u32(h0);
            h[b][1] = h2_as_u32(h1);
            if (LO) {
                lo[b][0] = h2_as_u32(__hfma2(u32_as_h2(b0), s0, __hneg2(h0)));
                lo[b][1] = h2_as_u32(__hfma2(u32_as_h2(b1), s1, __hneg2(h1)));
            }
        }
        uint32_t wv[4][L::D / 64];       // tokens t, t+4, t+8, t+12: the lane's 16 (8) channels
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *pv = rec + L::v_word(t + 4 * i, g, 0);
            if constexpr (L::D == 128) {
                const uint2 u = *reinterpret_cast<const uint2 *>(pv);
                wv[i][0] = u.x;
                wv[i][L::D / 64 - 1] = u.y;
            } else {
                wv[i][0] = *reinterpret_cast<const uint32_t *>(pv);
            }
        }
#pragma unroll
        for (int u = 0; u < L::D / 64; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = wv[i][u];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t sel = half ? 0x7632u : 0x5410u;
                uint32_t a01 = prmt(w[0], w[1], sel), a23 = prmt(w[2], w[3], sel);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int mt = 4 * u + 2 * half + i, b = mt * 16 / L::G;
                    mma16816(a.o[mt], a01 & M0, a01 & M1, a23 & M0, a23 & M1, h[b][0], h[b][1]);
                    if (LO)
                        mma16816(a.o[mt], a01 & M0, a01 & M1, a23 & M0, a23 & M1, lo[b][0],
                                 lo[b][1]);
                    a01 >>= 8;
                    a23 >>= 8;
                }
            }
        }
    }
}

// The open sequence's record to `dst` (m[8], l[8], o[8][D]).
template <typename L>
__device__ inline void put_record(float *dst, Acc<L> &a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float l = a.l[i];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
            dst[2 * t + i] = a.m[i];
            dst[8 + 2 * t + i] = l;
        }
        float z[L::NB];
#pragma unroll
        for (int b = 0; b < L::NB; ++b) z[b] = __shfl_sync(0xffffffffu, a.z[i], 4 * b + t);
        float *o = dst + 16 + (2 * t + i) * L::D;
#pragma unroll
        for (int mt = 0; mt < L::D / 16; ++mt) {
            const float zb = z[mt * 16 / L::G];
            o[16 * mt + g] = fmaf(a.o[mt][i], 16777216.f, -zb);       // rows g: c 2^-24
            o[16 * mt + 8 + g] = fmaf(a.o[mt][i + 2], 1048576.f, -zb);  // rows g + 8: c 2^-20
        }
    }
}

template <typename L>
__host__ __device__ constexpr int stage_bytes() { return 2 * L::REC; }
template <typename L>
__host__ __device__ constexpr int smem_bytes() {
    constexpr int ring = WARPS * NST * stage_bytes<L>();
    constexpr int comb = WARPS * rec_floats<L::D>() * 4;
    return (ring > comb ? ring : comb) + WARPS * NST * 8 + WARPS * 8;
}

template <typename L, int DT>
__global__ void __launch_bounds__(WARPS * 32, CTAS_PER_SM)
split_kernel(View v, Split p) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int RF = rec_floats<L::D>();
    constexpr int BODY = smem_bytes<L>() - WARPS * NST * 8 - WARPS * 8;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + BODY);
    int *owner = reinterpret_cast<int *>(smem + BODY + WARPS * NST * 8);   // run open at the end
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    uint8_t *ring = smem + wi * NST * stage_bytes<L>();
    uint64_t *bar = bars + wi * NST;
    if (lane < NST) mbar_init(bar + lane, 1);
    fence_mbar_init();
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    const int w = blockIdx.x * WARPS + wi;
    const int64_t total = units_of_all(v, p);
    const int64_t nw = warps_used(total, p.NW);
    int open = -1;
    bool dead = false;                      // a wait ran out
    Acc<L> acc;
    if (total > 0 && w < nw) {
        const int64_t u0 = unit_of(w, total, nw), u1 = unit_of(w + 1, total, nw);
        const int n = (int)(u1 - u0);
        Cursor c = seek(v, p, u0), ci = c;
        uint32_t masks = 0;                 // 2 bits a stage: the records on their way
        // Lane r knows record r of the 16 units from ci's at `base` on (of one run):
        // a unit's copies are issued by the two lanes that know its records.
        const uint8_t *src = nullptr;
        unsigned have = 0;
        int base = 0, left = 0;             // units that the lanes still know
        auto issue = [&](int slot) {        // the unit at ci into stage `slot`
            if (left == 0) {
                const int pos = ci.first + ci.u * UT + lane * RT;
                src = nullptr;
                if (pos < ci.len) {
                    src = record(v, ci.b, ci.sq / p.nhg, pos, L::REC);
                    if (src && !range_ok(v.status, src, L::REC, v.pool, v.n_pages * v.page_bytes))
                        src = nullptr;
                }
                have = __ballot_sync(0xffffffffu, src != nullptr);
                base = ci.u;
                left = min(16, ci.nu - ci.u);
            }
            const int k = ci.u - base;
            const unsigned two = have >> (2 * k) & 3u;
            // (a copy may be counted before its bytes are announced: the phase ends
            // with the announcement at the earliest)
            if (lane == 0) mbar_arrive_expect_tx(bar + slot, __popc(two) * L::REC + p.unsent);
            if ((lane >> 1) == k && src)
                bulk_g2s(ring + slot * stage_bytes<L>() + (lane & 1) * L::REC, src, L::REC, bar + slot);
            masks = (masks & ~(3u << (2 * slot))) | two << (2 * slot);
            --left;
            step(v, p, ci);
        };
        int issued = 0;
        for (; issued < NST && issued < n; ++issued) issue(issued);
        QFrag<L> q;
        acc_reset(acc);
        int cur = -1, slot = 0, parity = 0;
        int i = 0;
        for (; i < n; ++i) {
            const int run = c.b * p.nseq + c.sq;
            if (run != cur) {
                if (cur >= 0) {             // the last run ended inside this warp's units
                    float *dst = p.ws + ((int64_t)w + cur) * RF;
                    if (range_ok(v.status, dst, RF * 4, p.ws, p.ws_floats * 4)) put_record(dst, acc);
                    acc_reset(acc);
                }
                cur = run;
                load_q<L, DT>(v, p, c.b, c.sq, c.len, q);
            }
            dead = !warp_wait(bar + slot, parity);
            if (dead) break;
            const int pos = c.first + c.u * UT;
            const bool edge = pos + UT > c.len - p.nq + 1 ||
                              (p.q.window > 0 && pos < c.len - p.q.window);
            const int lo = p.q.window > 0 ? c.len - p.nq + 1 - p.q.window : 0;
            unit<L, DT == DKV_F16>(ring + slot * stage_bytes<L>(), masks >> (2 * slot) & 3, pos,
                                   edge, lo, c.len, p.q.window, q, acc);
            __syncwarp();
            if (issued < n) {
                issue(slot);
                ++issued;
            }
            step(v, p, c);
            if (++slot == NST) {
                slot = 0;
                parity ^= 1;
            }
        }
        open = dead ? -1 : cur;
        if (dead) {
            if (lane == 0) set_status(v.status, DKV_DEV_TIMEOUT);
            for (; i < issued; ++i) {       // the copies on their way, once more
                warp_wait(bar + slot, parity);
                if (++slot == NST) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
    }
    // Runs still open: warps of this CTA in the same run are joined by the
    // first of them.
    if (lane == 0) owner[wi] = open;
    // Every ring is idle now, but for one whose copies did not come: they may still
    // land where the records would stand, and the call's outputs are lost anyway.
    if (__syncthreads_or(dead)) return;
    float *recs = reinterpret_cast<float *>(smem);
    if (open >= 0) put_record(recs + wi * RF, acc);
    __syncthreads();
    for (int w0 = 0; w0 < WARPS;) {
        const int run = owner[w0];
        int w1 = w0 + 1;
        while (w1 < WARPS && owner[w1] == run) ++w1;
        if (run >= 0) {
            float *dst = p.ws + ((int64_t)blockIdx.x * WARPS + w0 + run) * RF;
            const bool ok = range_ok(v.status, dst, RF * 4, p.ws, p.ws_floats * 4);
            for (int i = threadIdx.x; i < 8 * L::D / 4 && ok; i += WARPS * 32) {
                const int h = i / (L::D / 4);
                float m = -INFINITY, l = 0.f;
                for (int k = w0; k < w1; ++k) m = fmaxf(m, recs[k * RF + h]);
                const float ref = m == -INFINITY ? 0.f : m;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = w0; k < w1; ++k) {
                    const float f = ex2(recs[k * RF + h] - ref);
                    const float4 y = reinterpret_cast<const float4 *>(recs + k * RF + 16)[i];
                    l = fmaf(recs[k * RF + 8 + h], f, l);
                    o.x = fmaf(y.x, f, o.x);
                    o.y = fmaf(y.y, f, o.y);
                    o.z = fmaf(y.z, f, o.z);
                    o.w = fmaf(y.w, f, o.w);
                }
                reinterpret_cast<float4 *>(dst + 16)[i] = o;
                if (i % (L::D / 4) == 0) {
                    dst[h] = m;
                    dst[8 + h] = l;
                }
            }
        }
        w0 = w1;
    }
}

// One block per run: joins its records.  Thread (head h, 4 channels).
template <int D, int DT>
__global__ void __launch_bounds__(8 * D / 4)
merge_kernel(View v, Split p) {
    constexpr int RF = rec_floats<D>();
    pdl_wait();
    pdl_trigger();
    const int run = blockIdx.x, b = run / p.nseq, sq = run - b * p.nseq;
    const int h = threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
    int64_t total, u0;
    int nu;
    units_around(v, p, b, &total, &u0, &nu);
    const int64_t nw = warps_used(total, p.NW);
    u0 += (int64_t)sq * nu;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nu > 0) {
        const int64_t u1 = u0 + nu;
        const int64_t wa = warp_of(u0, total, nw), wb = warp_of(u1 - 1, total, nw);
        // the warp that goes on to the next run left a record of its own; the others
        // of a CTA are in the record of its first one
        const bool closed = unit_of(wb + 1, total, nw) > u1;
        const int64_t last_open = closed ? wb - 1 : wb;
        const int open = last_open >= wa ? (int)(last_open / WARPS - wa / WARPS) + 1 : 0;
        const int n = open + (closed ? 1 : 0);
        constexpr int AT_ONCE = 8;         // loads on their way
        for (int k0 = 0; k0 < n; k0 += AT_ONCE) {
            float mr[AT_ONCE], lr[AT_ONCE];
            float4 y[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int k = k0 + i;
                const int64_t w = k >= open ? wb : k == 0 ? wa : (wa / WARPS + k) * WARPS;
                const float *r = p.ws + (w + run) * RF;
                mr[i] = -INFINITY;
                lr[i] = 0.f;
                y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < n && range_ok(v.status, r, RF * 4, p.ws, p.ws_floats * 4)) {
                    mr[i] = r[h];
                    lr[i] = r[8 + h];
                    y[i] = reinterpret_cast<const float4 *>(r + 16 + h * D)[c];
                }
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const float mx = fmaxf(m, mr[i]), ref = mx == -INFINITY ? 0.f : mx;
                const float f0 = ex2(m - ref), f1 = ex2(mr[i] - ref);
                l = fmaf(l, f0, lr[i] * f1);
                o.x = fmaf(o.x, f0, y[i].x * f1);
                o.y = fmaf(o.y, f0, y[i].y * f1);
                o.z = fmaf(o.z, f0, y[i].z * f1);
                o.w = fmaf(o.w, f0, y[i].w * f1);
                m = mx;
            }
        }
    }
    const int kvh = sq / p.nhg, hv = (sq - kvh * p.nhg) * 8 + h;
    if (hv >= p.nq * p.G) return;
    const int qt = hv / p.G, qh = kvh * p.G + hv - qt * p.G;
    const int64_t row = ((int64_t)b * p.nq + qt) * p.q.Hq + qh;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);    // NaN stays NaN
    const float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    uint2 u;
    if constexpr (DT == DKV_F16) {
        u = make_uint2(pack_h2(y[0], y[1]), pack_h2(y[2], y[3]));
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]);
        const __nv_bfloat162 d = __floats2bfloat162_rn(y[2], y[3]);
        u = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                       *reinterpret_cast<const uint32_t *>(&d));
    }
    reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.q.out) + row * D)[c] = u;
    if (p.q.lse && c == 0)
        p.q.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
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

int64_t runs(const View &v, int Hq, int nq) {
    const int nhg = (nq * (Hq / v.H) + 7) / 8;
    return (int64_t)v.B * v.H * nhg;
}

// CTAs of the split: all that the GPU holds, but no more than the cache's
// capacity gives MIN_UNITS a warp.
cudaError_t split_ctas(const View &v, int Hq, int nq, int *ctas) {
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t cap = ((int64_t)v.max_pages * v.page_size + UT - 1) / UT + 1;
    const int64_t most = (runs(v, Hq, nq) * cap + WARPS * MIN_UNITS - 1) / (WARPS * MIN_UNITS);
    *ctas = (int)(most < (int64_t)sms * CTAS_PER_SM ? most : (int64_t)sms * CTAS_PER_SM);
    return cudaSuccess;
}

template <typename L, int DT>
cudaError_t launch(const View &v, const Split &p, int ctas, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem_once(split_kernel<L, DT>, smem_bytes<L>(), &done);
    if (e == cudaSuccess)
        e = launch_pdl(split_kernel<L, DT>, dim3(ctas), dim3(WARPS * 32), smem_bytes<L>(), st, v, p);
    if (e == cudaSuccess)
        e = launch_pdl(merge_kernel<L::D, DT>, dim3((unsigned)(v.B * p.nseq)), dim3(8 * L::D / 4),
                       0, st, v, p);
    return e;
}

template <typename L>
cudaError_t launch_dt(const View &v, const Split &p, int ctas, cudaStream_t st) {
    return p.q.dtype == DKV_F16 ? launch<L, DKV_F16>(v, p, ctas, st)
                                : launch<L, DKV_BF16>(v, p, ctas, st);
}

}  // namespace

cudaError_t decode_workspace_floats(const View &v, int D, int Hq, int nq, int64_t *floats) {
    int ctas = 0;
    const cudaError_t e = split_ctas(v, Hq, nq, &ctas);
    if (e != cudaSuccess) return e;
    *floats = ((int64_t)ctas * WARPS + runs(v, Hq, nq)) * (16 + 8 * D);
    return cudaSuccess;
}

cudaError_t launch_decode(const View &v, int D, int G, const Query &q, int nq, float *ws,
                          int64_t ws_floats, int fault, cudaStream_t st) {
    Split p;
    p.q = q;
    p.nq = nq;
    p.G = q.Hq / v.H;
    p.nhg = (nq * p.G + 7) / 8;
    p.nseq = v.H * p.nhg;
    p.ws = ws;
    p.ws_floats = ws_floats;
    int ctas = 0;
    const cudaError_t e = split_ctas(v, q.Hq, nq, &ctas);
    if (e != cudaSuccess) return e;
    p.NW = ctas * WARPS;
    p.unsent = fault == 1 ? 16 : 0;
    if (D == 128)
        return G == 32 ? launch_dt<Lay<128, 32>>(v, p, ctas, st)
                       : launch_dt<Lay<128, 64>>(v, p, ctas, st);
    return G == 32 ? launch_dt<Lay<64, 32>>(v, p, ctas, st)
                   : launch_dt<Lay<64, 64>>(v, p, ctas, st);
}

}  // namespace kv4
}  // namespace dkv
