// host.h -- what the host sides of the C ABI share (defined in pa_api.cu): the
// argument checks, the per-device facts, the options and the caches of tensor maps.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/pa.h"
#include "kernels.h"

namespace pa {
namespace host {

int elem_bytes(int dtype);                      // 0: no pa_dtype
bool aligned(const void* p, uintptr_t a);       // and not null
int check_cache(const pa_cache_desc* c, PoolShape* shape);
int current_device();                           // -1: none
int* error_word(int dev);
int sm_count(int dev);
int option(int id);
unsigned long long wait_limit_ns();
int status_of(cudaError_t e);
// Encoded tensor maps from this thread's caches, or nullptr; valid until the next lookup.
const CUtensorMap* rows_map(const void* base, int dtype, int num_tokens, int num_heads, int head_dim,
                            int64_t token_stride, int box_heads, int box_tokens);
const CUtensorMap* group_map(const void* base, int dtype, const PoolShape& shape);

}  // namespace host
}  // namespace pa
