// kv4_write.cu -- the paged 4-bit cache: quantising tokens as they are
// written, and reading positions back.
//
// A warp takes a few tokens, one tensor of them, and all their heads: a token's
// sequence, page and record are found once.  D/8 lanes hold a row (one token,
// one kv head): a lane 8 neighbouring channels, which is one 16-byte access of
// a 16-bit input or output row and exactly one K word.  A block of 32 or 64
// channels is 4 or 8 neighbouring lanes, so its extremes take 2 or 3 shuffle
// steps.  A V word gathers one channel of each of 8 lanes (see
// kv4_common.cuh): an 8 x 8 transpose of nibbles in three shuffle steps.
//
// Measured on one B200: 21491 tokens of 8 heads (D 128, 16 bits) quantised in 44
// us: 196 instructions for 256 values in 72 % of the issue slots, 57 % of the
// ALU's, 6.9 warps a scheduler; no unit is full, and fewer instructions a value
// is what would help.  131072 tokens read as bf16 in 138 us, 5.0 TB/s in and out,
// bound by DRAM.
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_common.cuh"
#include "kv4_internal.h"

namespace dkv {
namespace kv4 {
namespace {

constexpr int WARPS = 8;

// 8 x 8 nibble transpose over 8 lanes: lane j's nibble g goes to lane g's nibble j.
__device__ inline uint32_t nib_transpose(uint32_t w) {
    const int lane = threadIdx.x & 31;
    uint32_t p = __shfl_xor_sync(0xffffffffu, w, 4);
    w = (lane & 4) ? (w & 0xFFFF0000u) | (p >> 16) : (w & 0x0000FFFFu) | (p << 16);
    p = __shfl_xor_sync(0xffffffffu, w, 2);
    w = (lane & 2) ? (w & 0xFF00FF00u) | ((p >> 8) & 0x00FF00FFu)
                   : (w & 0x00FF00FFu) | ((p & 0x00FF00FFu) << 8);
    p = __shfl_xor_sync(0xffffffffu, w, 1);
    w = (lane & 1) ? (w & 0xF0F0F0F0u) | ((p >> 4) & 0x0F0F0F0Fu)
                   : (w & 0x0F0F0F0Fu) | ((p & 0x0F0F0F0Fu) << 4);
    return w;
}

// 8 channels as they stand in memory.
template <int DT>
struct Raw {
    uint32_t u[DT == DKV_F32 ? 8 : 4];
};
template <int DT>
__device__ inline Raw<DT> load_raw(const void *p, int64_t i) {
    Raw<DT> x;
    const uint4 *q = reinterpret_cast<const uint4 *>(
        static_cast<const uint8_t *>(p) + i * (DT == DKV_F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (DT == DKV_F32 ? 2 : 1); ++k) {
        const uint4 a = __ldcs(q + k);
        x.u[4 * k] = a.x; x.u[4 * k + 1] = a.y; x.u[4 * k + 2] = a.z; x.u[4 * k + 3] = a.w;
    }
    return x;
}
template <int DT>
__device__ inline void to_float(const Raw<DT> &a, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if constexpr (DT == DKV_F32) x[k] = __uint_as_float(a.u[k]);
        else if constexpr (DT == DKV_F16) x[k] = (k & 1) ? h_hi(a.u[k / 2]) : h_lo(a.u[k / 2]);
        else x[k] = __uint_as_float((k & 1) ? a.u[k / 2] & 0xFFFF0000u : a.u[k / 2] << 16);
    }
}

__device__ inline float max_nan(float a, float b) {        // NaN if either is
    float c;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(c) : "f"(a), "f"(b));
    return c;
}
template <int DT>
__device__ inline uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t c;
    if constexpr (DT == DKV_F16) asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(c) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// The block's largest x and -x (at least 0); NaN if it holds one.
template <int DT, int LANES>
__device__ inline void extremes(const Raw<DT> &a, float *hi, float *nlo) {
    if constexpr (DT == DKV_F32) {
        float h = 0.f, n = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            h = max_nan(h, __uint_as_float(a.u[k]));
            n = fmaxf(n, -__uint_as_float(a.u[k]));
        }
#pragma unroll
        for (int o = 1; o < LANES; o *= 2) {
            h = max_nan(h, __shfl_xor_sync(0xffffffffu, h, o));
            n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
        }
        *hi = h;
        *nlo = n;
    } else {
        constexpr uint32_t SIGN = 0x80008000u;
        uint32_t h = max2_nan<DT>(max2_nan<DT>(a.u[0], a.u[1]), max2_nan<DT>(a.u[2], a.u[3]));
        uint32_t n = max2_nan<DT>(max2_nan<DT>(a.u[0] ^ SIGN, a.u[1] ^ SIGN),
                                  max2_nan<DT>(a.u[2] ^ SIGN, a.u[3] ^ SIGN));
        // both in one word: low half the largest, high half minus the smallest
        uint32_t m = max2_nan<DT>(max2_nan<DT>(prmt(h, n, 0x5410u), prmt(h, n, 0x7632u)), 0u);
#pragma unroll
        for (int o = 1; o < LANES; o *= 2)
            m = max2_nan<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
        if constexpr (DT == DKV_F16) {
            *hi = h_lo(m);
            *nlo = h_hi(m);
        } else {
            *hi = __uint_as_float(m << 16);
            *nlo = __uint_as_float(m & 0xFFFF0000u);
        }
    }
}

// Two fp32 operations in one instruction.
__device__ inline uint64_t f2(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ inline uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ inline uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Codes of 8 channels, channel i in nibble (i >> 1) + 4 (i & 1) for K, i for V;
// the quotients as in div7, two at a time.  rint(x / s) <= 15 - zero is code <=
// 15; code >= 0 holds by itself, as x >= lo and rint(lo / s) = -zero.  Adding
// 1.5 * 2^23 rounds to an integer in the low bits; the eight are put together
// with their offsets and those taken off at once.
template <bool K>
__device__ inline uint32_t encode8(const float (&x)[8], const Block &b) {
    const float top = (float)(15 - b.zero);
    const uint64_t r = f2(b.r, b.r), ms = f2(-b.s, -b.s);
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t a = f2(x[i], x[i + 1]);
        uint64_t q = mul2(a, r);
        q = fma2(fma2(ms, q, a), r, q);
        t[i] = __float_as_uint(__fadd_rn(fminf(__uint_as_float((uint32_t)q), top), 12582912.f));
        t[i + 1] = __float_as_uint(
            __fadd_rn(fminf(__uint_as_float((uint32_t)(q >> 32)), top), 12582912.f));
    }
    uint32_t w = 0;
#pragma unroll
    for (int n = 7; n >= 0; --n)
        w = w * 16u + t[K ? (n < 4 ? 2 * n : 2 * (n - 4) + 1) : n];
    return w - (0x4B400000u - (uint32_t)b.zero) * 0x11111111u;
}

// Record of `token` (head 0's; one head's pages are `head` bytes apart) and its
// place *tok there; nullptr if the token is to be skipped (before the first
// sequence or behind the last, a bad length, a bad page).  *b: a sequence at or
// before the token's.
__device__ inline uint8_t *token_record(const View &v, int token, int *b, int rec, int *tok) {
    if (v.starts) {
        while (*b < v.B && v.starts[*b + 1] <= token) ++*b;
    } else {
        *b = token / v.n_uniform;
    }
    if (*b >= v.B) return nullptr;
    const int s0 = seq_start(v, *b), n = (v.starts ? v.starts[*b + 1] : s0 + v.n_uniform) - s0;
    if (token < s0 || s0 < 0) return nullptr;      // before starts[0], or starts decrease
    const int len = seq_len(v, *b);
    if (len < 0) return nullptr;
    if (n > len) {                         // more rows than positions
        set_status(v.status, DKV_DEV_BAD_SEQLEN);
        return nullptr;
    }
    const int pos = len - n + (token - s0);
    *tok = pos & (RT - 1);
    return record(v, *b, 0, pos, rec);
}

constexpr int AHEAD = 4;     // rows' loads in flight per lane

template <typename L, int DT>
__global__ void __launch_bounds__(WARPS * 32)
append_kernel(View v, const void *K, const void *V, int64_t k_tok, int64_t k_head, int64_t v_tok,
              int64_t v_head, int per_warp, int heads) {
    constexpr int LG = L::D / 8, RW = 32 / LG;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, c8 = lane % LG;
    const int64_t w0 = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (w0 * per_warp >= v.n_rows) return;
    const int first = (int)(w0 * per_warp), last = min(v.n_rows, first + per_warp);
    if (w0 == 0 && blockIdx.y + blockIdx.z == 0) check_starts(v);
    const bool t = blockIdx.y;             // K, V
    const void *src = t ? V : K;
    const int64_t s_tok = t ? v_tok : k_tok, s_head = t ? v_head : k_head;
    const int64_t head_bytes = (int64_t)v.rpp * L::REC;
    const int hb = blockIdx.z * heads, he = min(v.H, hb + heads);      // this warp's heads
    int b = find_seq(v, first);
    for (int token = first; token < last; ++token) {
        if (v.starts)
            while (b < v.B && v.starts[b + 1] <= token) ++b;
        if (b >= v.B) break;               // padding
        Raw<DT> a[AHEAD];
        auto load = [&](int h0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (h0 + i * RW < he) {
                    a[i] = load_raw<DT>(src, token * s_tok + (h0 + i * RW) * s_head + c8 * 8);
                } else {
#pragma unroll
                    for (uint32_t &u : a[i].u) u = 0;
                }
            }
        };
        load(hb + lane / LG);              // on their way while the place is found
        int tok = 0;
        uint8_t *rec0 = token_record(v, token, &b, L::REC, &tok);
        if (!rec0) continue;
        // after the transpose lane g of each 8 holds chunk g of its half (u)
        const int off = t ? L::v_word(tok, c8 & 7, c8 >> 3)
                          : L::k_word(tok, (c8 & 3) * L::NJ + (c8 >> 2));
        const int blk = c8 / (L::G / 8);
        const int moff = c8 % (L::G / 8) ? -1 : t ? L::v_meta(tok, blk) : L::k_meta(tok, blk);
        for (int h0 = hb + lane / LG; h0 - lane / LG < he; h0 += AHEAD * RW) {
            if (h0 != hb + lane / LG) load(h0);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int head = h0 + i * RW;
                if (head - lane / LG >= he) break;             // no lane has one
                float x[8], hi, nlo;
                to_float<DT>(a[i], x);
                extremes<DT, L::G / 8>(a[i], &hi, &nlo);
                if (__any_sync(0xffffffffu, !(hi <= 32768.f && nlo <= 32768.f))) {
                    hi = nlo = 0.f;                             // NaN, infinite or too large
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[k] = clamp_in(x[k]);
                        hi = fmaxf(hi, x[k]);
                        nlo = fmaxf(nlo, -x[k]);
                    }
#pragma unroll
                    for (int o = 1; o < L::G / 8; o *= 2) {
                        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                        nlo = fmaxf(nlo, __shfl_xor_sync(0xffffffffu, nlo, o));
                    }
                }
                const Block q = block_rule(-nlo, hi);
                uint32_t w, m = q.meta;
                if (t) {
                    w = mirror_codes(nib_transpose(encode8<false>(x, q)), tok);
                    m = mirror_meta(m, tok);
                } else {
                    w = encode8<true>(x, q);
                }
                uint8_t *rec = rec0 + head * head_bytes;
                if (head < he &&
                    range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes)) {
                    *reinterpret_cast<uint32_t *>(rec + off) = w;
                    if (moff >= 0) *reinterpret_cast<uint16_t *>(rec + moff) = (uint16_t)m;
                }
            }
        }
    }
}

// (c - z) s of word w's 8 codes, nibble pairs (n, n + 4) to the output type.
// fp16: 1024 + c and 64 + c by masks, minus the same with z, times s: exact.
// bf16: 128 + c likewise (7 fraction bits); the product's 11 bits round once.
template <int DT>
__device__ inline void decode8(uint32_t w, uint32_t meta, uint32_t (&y)[DT == DKV_F32 ? 8 : 4]) {
    const uint32_t mm = meta | meta << 16;
    const __half2 s = meta_scale(mm);
    if constexpr (DT == DKV_BF16) {
        const __nv_bfloat162 sb = __float2bfloat162_rn(__low2float(s));
        const uint32_t zb = and_or<0x000F000Fu>(mm, 0x43004300u);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const uint32_t c = and_or<0x000F000Fu>(w >> (4 * n), 0x43004300u);
            const __nv_bfloat162 d = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&c),
                                                     *reinterpret_cast<const __nv_bfloat162 *>(&zb)),
                                             sb);
            y[n] = *reinterpret_cast<const uint32_t *>(&d);
        }
    } else {
        const __half2 z1024 = u32_as_h2(and_or<0x000F000Fu>(mm, 0x64006400u));
        const __half2 z64 = u32_as_h2(((mm << 4) & 0x00F000F0u) | 0x54005400u);
        const uint32_t w8 = w >> 8;
        const __half2 d[4] = {
            __hmul2(__hsub2(u32_as_h2(and_or<0x000F000Fu>(w, 0x64006400u)), z1024), s),
            __hmul2(__hsub2(u32_as_h2(and_or<0x00F000F0u>(w, 0x54005400u)), z64), s),
            __hmul2(__hsub2(u32_as_h2(and_or<0x000F000Fu>(w8, 0x64006400u)), z1024), s),
            __hmul2(__hsub2(u32_as_h2(and_or<0x00F000F0u>(w8, 0x54005400u)), z64), s)};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if constexpr (DT == DKV_F16) {
                y[n] = h2_as_u32(d[n]);
            } else {
                y[2 * n] = __float_as_uint(__low2float(d[n]));
                y[2 * n + 1] = __float_as_uint(__high2float(d[n]));
            }
        }
    }
}

template <typename L, int DT>
__global__ void __launch_bounds__(WARPS * 32)
read_kernel(View v, void *K, void *V, int per_warp, int heads) {
    constexpr int LG = L::D / 8, RW = 32 / LG;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, c8 = lane % LG;
    const int64_t w0 = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (w0 * per_warp >= v.n_rows) return;
    const int first = (int)(w0 * per_warp), last = min(v.n_rows, first + per_warp);
    if (w0 == 0 && blockIdx.y + blockIdx.z == 0) check_starts(v);
    const bool t = blockIdx.y;             // K, V
    uint8_t *dst = static_cast<uint8_t *>(t ? V : K);
    const int64_t head_bytes = (int64_t)v.rpp * L::REC;
    const int hb = blockIdx.z * heads, he = min(v.H, hb + heads);      // this warp's heads
    int b = find_seq(v, first);
    for (int token = first; token < last; ++token) {
        int tok = 0;
        const uint8_t *rec0 = token_record(v, token, &b, L::REC, &tok);
        if (!rec0) continue;
        const int blk = c8 / (L::G / 8);
        const int off = t ? L::v_word(tok, c8 & 7, c8 >> 3)
                          : L::k_word(tok, (c8 & 3) * L::NJ + (c8 >> 2));
        const int moff = t ? L::v_meta(tok, blk) : L::k_meta(tok, blk);
        for (int h0 = hb + lane / LG; h0 - lane / LG < he; h0 += AHEAD * RW) {
            uint32_t w[AHEAD], m[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int head = h0 + i * RW;
                const uint8_t *rec = rec0 + head * head_bytes;
                w[i] = m[i] = 0;
                if (head < he && range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes)) {
                    w[i] = *reinterpret_cast<const uint32_t *>(rec + off);
                    m[i] = *reinterpret_cast<const uint16_t *>(rec + moff);
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int head = h0 + i * RW;
                if (head - lane / LG >= he) break;             // no lane has one
                uint32_t x = w[i];
                if (t) {
                    // the 8 lanes share a token; channel i comes in nibble i and goes
                    // to nibble (i >> 1) + 4 (i & 1), as a K word has it
                    x = nib_transpose(mirror_codes(x, tok));
                    uint32_t e = x & 0x0F0F0F0Fu, o = (x >> 4) & 0x0F0F0F0Fu;   // even, odd channels
                    e = (e | e >> 4) & 0x00FF00FFu;
                    o = (o | o >> 4) & 0x00FF00FFu;
                    x = prmt(e, o, 0x6420u);
                }
                const uint32_t meta = t ? mirror_meta(m[i], tok) : m[i];
                uint32_t y[DT == DKV_F32 ? 8 : 4];
                decode8<DT>(x, meta, y);
                if (head >= he) continue;
                uint4 *q = reinterpret_cast<uint4 *>(
                    dst + (((int64_t)token * v.H + head) * L::D + c8 * 8) * (DT == DKV_F32 ? 4 : 2));
#pragma unroll
                for (int k = 0; k < (DT == DKV_F32 ? 2 : 1); ++k)
                    __stcs(q + k, make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
            }
        }
    }
}

// A warp's share: as many heads of a token as leave 2048 warps a tensor (a row of
// each of its lanes, AHEAD of them, all), and 2 or 4 tokens in long calls (a
// token's place is found once for its heads).  us of an append / a read, D 128,
// bf16, with one row, AHEAD rows and all heads:
//   8 heads,  256 tokens  2.9/2.6    3.7/2.9 (all)
//             512         3.8/3.7    3.7/2.8
//            1024         5.7/5.1    4.3/3.5
//            4096        18.4/14.5   9.4/6.3
//  32 heads,   64 tokens  3.1/2.9    3.7/3.1     8.4/5.3
//             128         3.9/3.9    3.9/3.1     8.4/5.3
//            1024        18.6/14.7   9.8/7.2    10.6/7.2
//            2048        35.6/27.4  17.4/11.5   16.4/11.3
// and of all 8 heads with 1, 2 and 4 tokens:
//            4096 tokens  9.4/6.3   10.2/7.6    11.9/8.4
//            8192        16.8/10.6  16.4/10.4   18.6/13.1
//           16384        31.9/19.7  30.9/18.2   31.3/18.6
//           65536       122/80.6   117/71.9    116/70.8
struct Share {
    int tokens, heads;
    dim3 grid;
};
template <typename L>
Share share_of(const View &v) {
    constexpr int RW = 32 / (L::D / 8);
    Share s;
    s.tokens = v.n_rows < 8192 ? 1 : v.n_rows < 16384 ? 2 : 4;
    s.heads = (int64_t)v.n_rows * v.H < 2048 * RW ? RW
              : v.n_rows < 2048 && v.H > AHEAD * RW ? AHEAD * RW : v.H;
    const int64_t per = (int64_t)WARPS * s.tokens;
    s.grid = dim3((unsigned)((v.n_rows + per - 1) / per), 2, (v.H + s.heads - 1) / s.heads);
    return s;
}

// Runs f.template operator()<Layout, dtype>() for the pool's layout.
template <typename F>
cudaError_t dispatch(int D, int G, int dtype, F f) {
#define DKV_KV4_DT(LAY)                                                   \
    (dtype == DKV_F32 ? f.template operator()<LAY, DKV_F32>()             \
     : dtype == DKV_F16 ? f.template operator()<LAY, DKV_F16>()           \
                        : f.template operator()<LAY, DKV_BF16>())
    using L12832 = Lay<128, 32>;
    using L12864 = Lay<128, 64>;
    using L6432 = Lay<64, 32>;
    using L6464 = Lay<64, 64>;
    if (D == 128) return G == 32 ? DKV_KV4_DT(L12832) : DKV_KV4_DT(L12864);
    return G == 32 ? DKV_KV4_DT(L6432) : DKV_KV4_DT(L6464);
#undef DKV_KV4_DT
}

struct AppendLaunch {
    const View &v;
    const void *K, *V;
    int64_t kt, kh, vt, vh;
    cudaStream_t st;
    template <typename L, int DT>
    cudaError_t operator()() const {
        const Share s = share_of<L>(v);
        return launch_pdl(append_kernel<L, DT>, s.grid, dim3(WARPS * 32), 0, st,
                          v, K, V, kt, kh, vt, vh, s.tokens,
                          s.heads);
    }
};
struct ReadLaunch {
    const View &v;
    void *K, *V;
    cudaStream_t st;
    template <typename L, int DT>
    cudaError_t operator()() const {
        const Share s = share_of<L>(v);
        return launch_pdl(read_kernel<L, DT>, s.grid, dim3(WARPS * 32), 0, st,
                          v, K, V, s.tokens, s.heads);
    }
};

}  // namespace

cudaError_t launch_append(const View &v, int D, int G, const void *K, const void *V, int dtype,
                          int64_t k_tok, int64_t k_head, int64_t v_tok, int64_t v_head,
                          cudaStream_t st) {
    return dispatch(D, G, dtype, AppendLaunch{v, K, V, k_tok, k_head, v_tok, v_head, st});
}

cudaError_t launch_read(const View &v, int D, int G, void *K, void *V, int dtype,
                        cudaStream_t st) {
    return dispatch(D, G, dtype, ReadLaunch{v, K, V, st});
}

}  // namespace kv4
}  // namespace dkv
