// kv4_internal.h -- host-side launchers of the paged 4-bit cache, between
// kv4_api.cu and the kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace dkv {
namespace kv4 {

struct View;

// K, V rows (token, head) at token * x_tok + head * x_head elements.
cudaError_t launch_append(const View &v, int D, int G, const void *K, const void *V, int dtype,
                          int64_t k_tok, int64_t k_head, int64_t v_tok, int64_t v_head,
                          cudaStream_t st);
cudaError_t launch_read(const View &v, int D, int G, void *K, void *V, int dtype,
                        cudaStream_t st);

// The queries of an attention call: row i, head h at i * tok + h * head elements of Q.
struct Query {
    const void *q;
    void *out;        // [rows][Hq][D] of the same type
    float *lse;       // [rows][Hq] or null
    int64_t tok, head;
    int dtype, Hq, window;
    float scale;
};

// Decode: nq query rows a sequence (rows b * nq + t).  fault: as dkv_debug_set_fault sets it.
cudaError_t decode_workspace_floats(const View &v, int D, int Hq, int nq, int64_t *floats);
cudaError_t launch_decode(const View &v, int D, int G, const Query &q, int nq, float *ws,
                          int64_t ws_floats, int fault, cudaStream_t st);

// Prompt: ragged query rows (v.starts, v.n_rows), or the same number each.
cudaError_t prompt_workspace_floats(const View &v, int D, int Hq, int64_t *floats);
cudaError_t launch_prompt(const View &v, int D, int G, const Query &q, float *ws,
                          int64_t ws_floats, cudaStream_t st);

}  // namespace kv4
}  // namespace dkv
