// kv4_write.cu -- the paged 4-bit cache: quantising tokens as they are
// written, and reading positions back.
//
// Both directions take D/8 lanes a row (one token, one kv head, one tensor):
// a lane holds 8 neighbouring channels, which is one 16-byte access of a
// 16-bit input or output row and exactly one K word.  A block of 32 or 64
// channels is 4 or 8 neighbouring lanes, so its extremes take 2 or 3 shuffle
// steps.  A V word gathers one channel of each of 8 lanes (see
// kv4_common.cuh): an 8 x 8 transpose of nibbles in three shuffle steps.
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

template <int DT>
__device__ inline void load8(const void *p, int64_t i, float (&x)[8]) {
    if constexpr (DT == DKV_F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = q[0], b = q[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == DKV_F16) {
                x[2 * k] = h_lo(u[k]);
                x[2 * k + 1] = h_hi(u[k]);
            } else {
                x[2 * k] = __uint_as_float(u[k] << 16);
                x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
            }
        }
    }
}

template <int DT>
__device__ inline void store8(void *p, int64_t i, const float (&x)[8]) {
    if constexpr (DT == DKV_F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == DKV_F16) {
                u[k] = pack_h2(x[2 * k], x[2 * k + 1]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
                u[k] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
            make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// Where row `row` = (token, head) of the call lives: the record and the token
// in it; nullptr if the row is to be skipped (behind the last sequence, a bad
// length, a bad page).  first: the warp's first token, b0 its sequence.
__device__ inline uint8_t *row_record(const View &v, int token, int head, int b0, int rec,
                                      int *tok) {
    int b = b0;
    if (v.starts) {
        while (b < v.B && v.starts[b + 1] <= token) ++b;
    } else {
        b = token / v.n_uniform;
    }
    if (b >= v.B) return nullptr;
    const int s0 = seq_start(v, b), n = (v.starts ? v.starts[b + 1] : s0 + v.n_uniform) - s0;
    if (token < s0 || s0 < 0) {            // starts decrease, or begin behind a row
        set_status(v.status, DKV_DEV_BAD_SEQLEN);
        return nullptr;
    }
    const int len = seq_len(v, b);
    if (len < 0) return nullptr;
    if (n > len) {                         // more rows than positions
        set_status(v.status, DKV_DEV_BAD_SEQLEN);
        return nullptr;
    }
    const int pos = len - n + (token - s0);
    *tok = pos & (RT - 1);
    return record(v, b, head, pos, rec);
}

template <typename L, int DT>
__global__ void __launch_bounds__(WARPS * 32)
append_kernel(View v, const void *K, const void *V, int64_t k_tok, int64_t k_head, int64_t v_tok,
              int64_t v_head) {
    constexpr int LG = L::D / 8, RW = 32 / LG;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, c8 = lane % LG;
    const int64_t r0 = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RW;
    const int64_t rows = (int64_t)v.n_rows * v.H;
    if (r0 >= rows) return;
    if (r0 == 0 && blockIdx.y == 0) check_starts(v);
    const int b0 = find_seq(v, (int)(r0 / v.H));
    const int64_t r = min(r0 + lane / LG, rows - 1);   // lanes of a missing row repeat the last
    const bool have = r0 + lane / LG < rows;
    const int token = (int)(r / v.H), head = (int)(r - (int64_t)token * v.H);
    const int t = blockIdx.y;
    float x[8];
    if (t == 0) load8<DT>(K, token * k_tok + head * k_head + c8 * 8, x);
    else load8<DT>(V, token * v_tok + head * v_head + c8 * 8, x);
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = clamp_in(x[i]);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < L::G / 8; o *= 2) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const Block blk = block_rule(lo, hi);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w |= (uint32_t)block_code(blk, x[i]) << (4 * (t == 0 ? (i >> 1) + 4 * (i & 1) : i));
    if (t) w = nib_transpose(w);
    int tok = 0;
    uint8_t *rec = have ? row_record(v, token, head, b0, L::REC, &tok) : nullptr;
    if (!rec || !range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes)) return;
    // after the transpose lane g of each 8 holds chunk g of its half (u)
    const int off = t == 0 ? L::k_word(tok, (c8 & 3) * L::NJ + (c8 >> 2))
                           : L::v_word(tok, c8 & 7, c8 >> 3);
    *reinterpret_cast<uint32_t *>(rec + off) = t == 0 ? w : mirror_codes(w, tok);
    if (c8 % (L::G / 8) == 0) {
        const int b = c8 / (L::G / 8);
        *reinterpret_cast<uint16_t *>(rec + (t == 0 ? L::k_meta(tok, b) : L::v_meta(tok, b))) =
            (uint16_t)(t == 0 ? blk.meta : mirror_meta(blk.meta, tok));
    }
}

template <typename L, int DT>
__global__ void __launch_bounds__(WARPS * 32)
read_kernel(View v, void *K, void *V) {
    constexpr int LG = L::D / 8, RW = 32 / LG;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, c8 = lane % LG;
    const int64_t r0 = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RW;
    const int64_t rows = (int64_t)v.n_rows * v.H;
    if (r0 >= rows) return;
    if (r0 == 0 && blockIdx.y == 0) check_starts(v);
    const int b0 = find_seq(v, (int)(r0 / v.H));
    const int64_t r = r0 + lane / LG;
    const int token = (int)(r / v.H), head = (int)(r - (int64_t)token * v.H);
    const int t = blockIdx.y;
    int tok = 0;
    uint8_t *rec = r < rows ? row_record(v, token, head, b0, L::REC, &tok) : nullptr;
    if (rec && !range_ok(v.status, rec, L::REC, v.pool, v.n_pages * v.page_bytes)) rec = nullptr;
    uint32_t w = 0, m = 0;
    if (rec) {
        const int b = c8 / (L::G / 8);
        w = *reinterpret_cast<const uint32_t *>(
            rec + (t == 0 ? L::k_word(tok, (c8 & 3) * L::NJ + (c8 >> 2))
                          : L::v_word(tok, c8 & 7, c8 >> 3)));
        m = *reinterpret_cast<const uint16_t *>(
            rec + (t == 0 ? L::k_meta(tok, b) : L::v_meta(tok, b)));
    }
    if (t) {
        w = nib_transpose(mirror_codes(w, tok));      // the 8 lanes share a token
        m = mirror_meta(m, tok);
    }
    if (!rec) return;
    const float s = __half2float(__ushort_as_half((unsigned short)(m & 0xFFF0u)));
    const int zero = (int)(m & 0xFu);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = t == 0 ? (i >> 1) + 4 * (i & 1) : i;
        x[i] = (float)((int)((w >> (4 * n)) & 15u) - zero) * s;     // exact (<= 11 bits)
    }
    store8<DT>(t == 0 ? K : V, r * L::D + c8 * 8, x);
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
        const int64_t per = (int64_t)WARPS * (32 / (L::D / 8));
        const int64_t blocks = ((int64_t)v.n_rows * v.H + per - 1) / per;
        return launch_pdl(append_kernel<L, DT>, dim3((unsigned)blocks, 2), dim3(WARPS * 32), 0, st,
                          v, K, V, kt, kh, vt, vh);
    }
};
struct ReadLaunch {
    const View &v;
    void *K, *V;
    cudaStream_t st;
    template <typename L, int DT>
    cudaError_t operator()() const {
        const int64_t per = (int64_t)WARPS * (32 / (L::D / 8));
        const int64_t blocks = ((int64_t)v.n_rows * v.H + per - 1) / per;
        return launch_pdl(read_kernel<L, DT>, dim3((unsigned)blocks, 2), dim3(WARPS * 32), 0, st,
                          v, K, V);
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
