// kv4_common.cuh -- layout of the paged 4-bit cache (dkv_kv4_*), its block
// rule, and the device views its kernels share.
//
// A page holds page_size positions of one sequence for every kv head, as
// records of 16 positions: record (h, r) at page + (h * page_size/16 + r) *
// REC.  A record is
//   [K codes 16 x D/2][V codes 16 x D/2][K meta 16 x NB x 2][V meta 16 x NB x 2]
// with NB = D / group blocks a token.  It is one contiguous bulk copy (every
// size is a multiple of 16 B), and inside it codes and meta stand where the
// decode kernel's tensor-core fragments want them, so that a lane's part of a
// fragment is one wide shared-memory load without bank conflicts:
//  K codes: a token's row of D/8 words stands in row slot k_slot(token); word
//   t * (D/32) + j holds channels 32j + 8t .. + 7, channel 8t + i of it in
//   nibble (i >> 1) + 4 (i & 1): masks 0x000F000F / 0x00F000F0 then give pairs
//   of neighbouring channels, the two halves of an fp16x2 operand.
//  V codes: channel 16 mt + 8 e + g is nibble 2 (mt % 4) + e of word mt / 4 of
//   chunk g: rows g and g + 8 of the 16-channel tile mt.
//  K meta: halfword token * NB + block.
//  V meta: halfword ((token % 4) * NB + block) * 4 + token / 4.
// A meta halfword is the block's scale as fp16 -- 7 significant bits, so its
// low 4 bits are zero -- with the zero point (0..15) in those 4 bits.  The
// value held, (code - zero) * scale, has at most 4 + 7 significant bits and is
// exact in fp16; so is zero * scale.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/dkv.h"
#include "dkv_common.cuh"

namespace dkv {
namespace kv4 {

constexpr int RT = 16;    // positions per record

template <int D_, int G_>
struct Lay {
    static constexpr int D = D_, G = G_, NB = D_ / G_;
    static constexpr int NJ = D_ / 32;             // 32-channel chunks
    static constexpr int ROW = D_ / 2;             // bytes of one token's codes
    static constexpr int OFF_V = RT * ROW;
    static constexpr int OFF_KM = 2 * RT * ROW;
    static constexpr int OFF_VM = OFF_KM + RT * NB * 2;
    static constexpr int REC = OFF_VM + RT * NB * 2;
    static_assert(REC % 16 == 0 && OFF_KM % 16 == 0 && OFF_VM % 16 == 0, "bulk copies, wide loads");

    // The K tile's MMA rows g and g + 1 are tokens 4 apart; their rows land in
    // different halves (D = 128) or quarters (D = 64) of the banks.
    __host__ __device__ static int k_slot(int tok) {
        return D_ == 128 ? tok ^ ((tok >> 2) & 1) : tok ^ (((tok >> 2) & 1) << 1);
    }
    // byte of K word w (0 .. D/8-1) of a token, from the record's start
    __host__ __device__ static int k_word(int tok, int w) { return k_slot(tok) * ROW + w * 4; }
    // byte of word u of chunk g (0..7) of a token's V codes
    __host__ __device__ static int v_word(int tok, int g, int u) {
        return OFF_V + tok * ROW +
               (D_ == 128 ? (g ^ (((tok >> 1) & 1) << 2)) * 8 + u * 4 : g * 4);
    }
    __host__ __device__ static int k_meta(int tok, int b) { return OFF_KM + (tok * NB + b) * 2; }
    __host__ __device__ static int v_meta(int tok, int b) {
        return OFF_VM + (((tok & 3) * NB + b) * 4 + (tok >> 2)) * 2;
    }
};

inline int rec_bytes(int head_dim, int group) {
    return 2 * RT * (head_dim / 2) + 2 * RT * (head_dim / group) * 2;
}

// The pool and the sequences of one call, by value to the kernels.
struct View {
    uint8_t *pool;
    int64_t n_pages, page_bytes;
    int32_t *status;
    int32_t H, page_size, rpp;     // rpp: records per page (and head)
    const int32_t *table;          // [B][max_pages]
    const int32_t *lens;           // [B]
    const int32_t *starts;         // [B + 1], or null: n_uniform rows a sequence
    int32_t B, max_pages;
    int32_t n_rows, n_uniform;
};

__device__ inline int seq_start(const View &v, int b) {
    return v.starts ? v.starts[b] : b * v.n_uniform;
}

// One warp of a grid looks all starts over.
__device__ inline void check_starts(const View &v) {
    if (!v.starts) return;
    for (int b = threadIdx.x & 31; b < v.B; b += 32)
        if (v.starts[b] < 0 || v.starts[b + 1] < v.starts[b])
            set_status(v.status, DKV_DEV_BAD_SEQLEN);
}

// Length of sequence b; < 0 (and DKV_DEV_BAD_SEQLEN) if it lies outside the
// block table.
__device__ inline int seq_len(const View &v, int b) {
    const int n = v.lens[b];
    if (n < 0 || (int64_t)n > (int64_t)v.max_pages * v.page_size) {
        set_status(v.status, DKV_DEV_BAD_SEQLEN);
        return -1;
    }
    return n;
}

// Record holding position pos (a multiple of 16 or any position in it) of
// sequence b, kv head h; nullptr (and DKV_DEV_BAD_PAGE) for a table entry
// outside the pool.  The caller has checked pos against the table's width.
__device__ inline uint8_t *record(const View &v, int b, int h, int pos, int rec) {
    const int pi = pos / v.page_size;
    const int page = v.table[(int64_t)b * v.max_pages + pi];
    if (page < 0 || page >= v.n_pages) {
        set_status(v.status, DKV_DEV_BAD_PAGE);
        return nullptr;
    }
    const int r = (pos - pi * v.page_size) / RT;
    return v.pool + (int64_t)page * v.page_bytes + ((int64_t)h * v.rpp + r) * rec;
}

// Sequence that row i of a ragged batch belongs to: the number of sequences
// that end at or before i (a whole warp asks, all lanes for the same i).
// Returns B for a row behind the last sequence.
__device__ inline int find_seq(const View &v, int i) {
    if (!v.starts) return i / v.n_uniform;
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int j0 = 1; j0 <= v.B; j0 += 32) {
        const int j = j0 + lane;
        const bool past = j <= v.B && v.starts[j] <= i;
        n += __popc(__ballot_sync(0xffffffffu, past));
    }
    return n;
}

// ---------------------------------------------------------------------------
// The block rule.  lo <= 0 <= hi: the block's extremes with 0 among them.
// ---------------------------------------------------------------------------
struct Block {
    float s, r;        // scale and about its reciprocal (1 for an all-zero block)
    int zero;
    uint16_t meta;
};

__device__ inline float clamp_in(float x) {
    // NaN counts as 0; fmaxf/fminf drop a NaN operand, so it is taken out first
    x = x != x ? 0.f : x;
    return fminf(fmaxf(x, -32768.f), 32768.f);
}

// RN(x / s) for s of at most 7 significant bits and r within 1 ulp of 1 / s, as
// far as rint() of it can tell.  q0 = RN(x r) is within 2.5 ulp, so x - s q0 has
// few bits and the first FMA is exact; the second is RN of x / s + d, |d| <=
// 2.5 * 2^-23 ulp.  x / s is never the midpoint of two floats (25 bits times an
// odd factor of s is no 24-bit x) and lies at least 2^-8 ulp away from one, so d
// cannot matter.  Quotients whose steps underflow are far below 1/2.
__device__ inline float div7(float x, float s, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-s, q, x), r, q);
}

__device__ inline Block block_rule(float lo, float hi) {
    const float r = __fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f);
    // up to 7 significant bits; below 2^-14 (fp16's subnormals) to a multiple of 2^-20
    float s = __uint_as_float((__float_as_uint(r) + 0x1FFFFu) & ~0x1FFFFu);
    if (r < 6.103515625e-05f) s = ceilf(r * 1048576.0f) * 9.5367431640625e-07f;
    Block b;
    const bool none = !(s > 0.f);
    b.s = none ? 1.f : s;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(b.r) : "f"(b.s));
    // rint by adding 1.5 * 2^23; at most 15, as s >= r
    const float z = __fadd_rn(div7(-lo, b.s, b.r), 12582912.f);
    b.zero = min(15, (int)(__float_as_uint(z) - 0x4B400000u));
    b.meta = (uint16_t)(__half_as_ushort(__float2half_rn(s)) | b.zero);
    return b;
}
// An all-zero block (meta 0) takes s = 1, zero = 0: its elements are 0 or so
// small that their range underflows, and their codes come out 0.

// The V codes and meta of odd positions are stored mirrored, 15 - c with 15 - z
// and -s: the same value, (c - z) s.  The tensor cores cut sums towards zero;
// with every other sum of products turned around, the cuts do not add up.
// Mirror of a V word / V meta halfword at position tok (its own inverse).
__device__ inline uint32_t mirror_codes(uint32_t w, int tok) { return (tok & 1) ? ~w : w; }
__device__ inline uint32_t mirror_meta(uint32_t m, int tok) { return (tok & 1) ? m ^ 0x800Fu : m; }

__device__ inline __half2 meta_scale(uint32_t m) { return u32_as_h2(m & 0xFFF0FFF0u); }
// zero points of two blocks as exact fp16 integers
__device__ inline __half2 meta_zero(uint32_t m) {
    return __hsub2(u32_as_h2((m & 0x000F000Fu) | 0x64006400u), u32_as_h2(0x64006400u));
}

// A bounded wait whose outcome the whole warp shares: each lane has a clock of
// its own to give up by, and what follows a wait takes all lanes.
__device__ inline bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

// Lets KERNEL have `bytes` of dynamic shared memory on the current device; the
// attribute belongs to the device's copy of the kernel and is set once for each.
template <typename Kernel>
inline cudaError_t allow_smem_once(Kernel *kernel, int bytes, std::atomic<uint64_t> *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace kv4
}  // namespace dkv
