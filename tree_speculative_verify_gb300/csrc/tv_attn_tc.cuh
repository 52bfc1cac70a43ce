// tcgen05 tensor-core tree-verify attention (bf16, d = 512): host-side interface.
#pragma once

#include <cuda.h>

#include "tv_attn_common.cuh"

// True when the tensor-core kernel takes this shape (bf16, d = 512, D <= 8, B <= 12288; a C4
// selection list is gathered into the workspace first).
bool tv_tc_shape_ok(const tv_shape* s);
// True when the tensor-core kernel is compiled in and the current device can run it.
bool tv_tc_available();
// Workspace bytes the tensor-core kernel needs for this shape.
size_t tv_tc_workspace_size(const tv_shape* s);
// Enqueue the tensor-core kernel (and its merge) on `stream`.
int tv_launch_attn_tc(const tv_shape* s, const tv::AttnParams<__nv_bfloat16>& p, void* workspace,
                      cudaStream_t stream);

// The same for tv_chunk_attn (bf16, d = 512).
size_t tv_chunk_tc_workspace(const tv_shape* s);
int tv_launch_chunk_tc(const tv_shape* s, int n_new, const int32_t* starts, const void* Q,
                       const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                       const void* rawK, const void* rawV, const int32_t* L, float scale, void* O,
                       float* lse, void* workspace, int32_t* status, cudaStream_t stream);

// The same for batches of few new tokens per request (bf16, d a multiple of 128).
bool tv_few_ok(const tv_shape* s);
size_t tv_few_workspace(const tv_shape* s, int n_new);
int tv_launch_few(const tv_shape* s, int n_new, const int32_t* starts, const void* Q,
                  const void* c4K, const void* c4V, const void* c128K, const void* c128V,
                  const void* rawK, const void* rawV, const int32_t* L, float scale, void* O,
                  float* lse, void* workspace, int32_t* status, cudaStream_t stream);

// Shared by the two: the C128 entries of paged pools copied to contiguous rows (K, then V), their rows
// per request and bytes of one of K / V (0: not needed); tensor maps; the test aid's settings.
int64_t tv_chunk_c128_stride(const tv_shape* s);
size_t tv_chunk_gather_bytes(const tv_shape* s);
int tv_chunk_gather(const tv_shape* s, const int32_t* starts, const int32_t* L, const void* c128K,
                    const void* c128V, void* rows, int32_t* status, cudaStream_t stream);
bool tv_make_map(CUtensorMap* m, const void* base, int rank, int d, uint64_t rows, uint64_t batch,
                 uint32_t box_rows);
void tv_attn_test_aid(uint64_t* timeout_ns, int* withhold_tile);
