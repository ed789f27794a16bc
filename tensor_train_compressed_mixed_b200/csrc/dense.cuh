// The handle of a dense table: its lookup and gradient (dense.cu), and its projection (project.cu).
#pragma once

#include "matmul.cuh"

struct tt_emb_dense_handle {
    int64_t rows = 0, pad = -1;
    int dim = 0, table_type = TT_F32, grad_type = TT_F32;
    float scale = 1.f;
    const void* table = nullptr;
    void* grad = nullptr;
    char* ws = nullptr;
    int64_t ws_n = -1;
    char* project_ws = nullptr;
    size_t project_bytes = 0;
    tt::MatmulFits fits;         // of the handle's device, asked for by the first call that wants them
    bool has_fits = false;
    int32_t* d_status = nullptr;
    int device = 0, num_sms = 148;
    bool clusters = false;       // one of k_token_sort fits this device
    cudaStream_t last_stream = nullptr;
    bool used_stream = false;
    int last_error = TT_OK;
    int inject = TT_INJECT_NONE;     // tt_emb_dense_debug_inject, armed until a product on the tensor cores takes it
};

namespace tt {

// records a failed call on the handle
inline int note(tt_emb_dense_t h, int rc)
{
    if (h && rc != TT_OK) h->last_error = rc;
    return rc;
}

// the handle's device is current
inline int ready(tt_emb_dense_t h)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TT_ERR_CUDA;
    return dev == h->device ? TT_OK : TT_ERR_STATE;
}

}  // namespace tt
