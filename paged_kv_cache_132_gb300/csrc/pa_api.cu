// pa_api.cu -- the C ABI declared in include/pa.h: argument checks, the
// per-device error word, the library options, the partition choice, and the
// launches.
//
// Every argument error is caught here, before anything reaches the GPU; the
// kernels only report what depends on device data (ids, slots, lengths) or on
// time (a bounded wait that ran out), through the error word.
//
// Host cost per call is kept small because decode runs once per layer per
// step: per-device facts (error word address, SM count) are looked up once
// and then read with atomic loads, options are atomics initialised once from
// the environment, and the TMA descriptors of the pools are encoded once per
// (pool, shape) and cached per host thread.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "../../include/pa.h"
#include "host.h"
#include "kernels.h"

namespace {

// One error word per device (a __device__ variable exists once per device
// that loads the library); read and cleared by pa_get_device_error.
__device__ int g_device_error;

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
std::atomic<int*> g_error_ptr[kMaxDevices];
std::atomic<int> g_sm_count[kMaxDevices];

int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    return dev;
}

int* error_word(int dev) {
    int* p = g_error_ptr[dev].load(std::memory_order_acquire);
    if (p) return p;
    std::lock_guard<std::mutex> lock(g_mutex);
    p = g_error_ptr[dev].load(std::memory_order_relaxed);
    if (!p) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_device_error) != cudaSuccess) return nullptr;
        p = static_cast<int*>(a);
        g_error_ptr[dev].store(p, std::memory_order_release);
    }
    return p;
}

int l2_bytes(int dev) {
    static std::atomic<int> cached[kMaxDevices];
    int n = cached[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrL2CacheSize, dev) != cudaSuccess || n <= 0) return 0;
    cached[dev].store(n, std::memory_order_release);
    return n;
}

int sm_count(int dev) {
    int n = g_sm_count[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
    g_sm_count[dev].store(n, std::memory_order_release);
    return n;
}

// ---- library options ---------------------------------------------------------
constexpr int kNumOptions = 3;
std::atomic<int> g_option[kNumOptions];
std::once_flag g_option_env_once;

bool env_is(const char* name, const char* value) {
    const char* v = std::getenv(name);
    return v && std::strcmp(v, value) == 0;
}

int option(int id) {
    std::call_once(g_option_env_once, [] {
        g_option[PA_OPT_DEBUG_CHECKS].store(env_is("PA_DEBUG_CHECKS", "1") ? 1 : 0);
        g_option[PA_OPT_DECODE_KERNEL].store(env_is("PA_DECODE_KERNEL", "simt") ? 1 : 0);
        g_option[PA_OPT_DROP_FIRST_FILL].store(env_is("PA_DEBUG_DROP_FIRST_FILL", "1") ? 1 : 0);
    });
    return g_option[id].load(std::memory_order_relaxed);
}

// An NVTX range around each entry point (free when no tool is attached).
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

// Wall-time limit of every wait inside a kernel (environment variable
// PA_WAIT_TIMEOUT_MS, default 2000 ms).
unsigned long long wait_limit_ns() {
    static const unsigned long long limit = [] {
        const char* s = std::getenv("PA_WAIT_TIMEOUT_MS");
        long long ms = s ? std::atoll(s) : 2000;
        if (ms <= 0) ms = 2000;
        return (unsigned long long)ms * 1000000ull;
    }();
    return limit;
}

int elem_bytes(int dtype) {
    switch (dtype) {
        case PA_F32: return 4;
        case PA_F16:
        case PA_BF16: return 2;
        default: return 0;
    }
}

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache(const pa_cache_desc* c, pa::PoolShape* shape) {
    if (!c) return PA_ERR_INVALID_ARG;
    const int eb = elem_bytes(c->dtype);
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->block_size <= 0 || c->head_dim <= 0 || eb == 0)
        return PA_ERR_INVALID_ARG;
    if (((int64_t)c->head_dim * eb) % 16 != 0) return PA_ERR_INVALID_ARG;
    shape->num_blocks = c->num_blocks;
    shape->num_kv_heads = c->num_kv_heads;
    shape->block_size = c->block_size;
    shape->head_dim = c->head_dim;
    shape->elem_bytes = eb;
    return PA_OK;
}

int max_parts_for(int max_context_len, int partition) {
    const int parts = (max_context_len + partition - 1) / partition;
    return parts < 1 ? 1 : parts;
}

bool partition_ok(int32_t partition_size) { return partition_size == 0 || (partition_size > 0 && partition_size % 64 == 0); }

// cuTensorMapEncodeTiled, fetched through the runtime so that the library
// does not link against the driver library directly.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// The pool [NB][Hkv][B][d] as a 2-D tensor of NB*Hkv*B rows of d 16-bit
// elements; a box is 64 elements (128 bytes, the swizzle span) x B rows.
// With interleave (the decode kernel, head_dim 128 and 8- or 16-token blocks) the
// view is 3-D instead, one box per (block, head) tile.
bool encode_pool_map(CUtensorMap* map, const void* base, int dtype, const pa::PoolShape& shape,
                     bool interleave = true) {
    const int64_t rows = shape.num_blocks * shape.num_kv_heads * shape.block_size;
    if (rows <= 0 || rows >= (1LL << 31) || shape.head_dim % 64 != 0) return false;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const CUtensorMapDataType type =
        dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    std::memset(map, 0, sizeof(*map));
    CUresult r;
    if (interleave && pa::interleaved_stage(shape.head_dim, shape.block_size)) {
        // [rows][2 slabs][64]: one box = one whole (block, head) tile.
        const cuuint64_t dims[3] = {64, 2, (cuuint64_t)rows};
        const cuuint64_t strides[2] = {128, 256};
        const cuuint32_t box[3] = {64, 2, (cuuint32_t)shape.block_size};
        const cuuint32_t elem_strides[3] = {1, 1, 1};
        r = encode(map, type, 3, const_cast<void*>(base), dims, strides, box, elem_strides,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        // [rows][d]: one box = one 64-element column slab of a tile.
        const cuuint64_t dims[2] = {(cuuint64_t)shape.head_dim, (cuuint64_t)rows};
        const cuuint64_t strides[1] = {(cuuint64_t)shape.head_dim * 2};
        const cuuint32_t box[2] = {64, (cuuint32_t)shape.block_size};
        const cuuint32_t elem_strides[2] = {1, 1};
        r = encode(map, type, 2, const_cast<void*>(base), dims, strides, box, elem_strides,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS;
}

// The pool's rows in groups of eight, as a 4-D tensor {64, 8 rows, d / 64 slabs,
// groups}: one box = one (block, head) tile, the slabs of 8 rows side by side in shared
// memory (the tree attention's K and V tiles).
bool encode_group_map(CUtensorMap* map, const void* base, int dtype, const pa::PoolShape& shape) {
    const int64_t rows = shape.num_blocks * shape.num_kv_heads * shape.block_size;
    if (rows <= 0 || rows >= (1LL << 31) || shape.head_dim % 64 != 0 || shape.block_size % 8 != 0) return false;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const CUtensorMapDataType type =
        dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    std::memset(map, 0, sizeof(*map));
    const cuuint64_t row = (cuuint64_t)shape.head_dim * 2;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)shape.head_dim / 64, (cuuint64_t)rows / 8};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)shape.head_dim / 64, (cuuint32_t)shape.block_size / 8};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    return encode(map, type, 4, const_cast<void*>(base), dims, strides, box, elem_strides,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [num_tokens][num_heads][d] of 16-bit elements, `token_stride` elements
// from token to token, as a 3-D tensor {d, heads, tokens}; a box is 64 elements
// x box_heads heads x box_tokens tokens, 128 bytes per (token, head) row.
bool encode_rows_map(CUtensorMap* map, const void* base, int dtype, int num_tokens, int num_heads, int head_dim,
                     int64_t token_stride, int box_heads, int box_tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode || head_dim % 64 != 0) return false;
    const CUtensorMapDataType type =
        dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    std::memset(map, 0, sizeof(*map));
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)num_heads, (cuuint64_t)num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    return encode(map, type, 3, const_cast<void*>(base), dims, strides, box, elem_strides,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Cache of encoded tensor maps, per host thread (no lock).  An encoding is a
// pure function of its key (base address, shape, dtype, view), so a cached
// map is valid for as long as the key matches, whatever the caller did with
// the memory in between.  Kernel parameters are copied at launch, so the
// returned pointer is only used before the next lookup on this thread.  Rows of
// activations have a cache of their own: new ones come with every call, and would
// put the pools' maps out, which stay for the life of a server.
struct MapKey {
    int kind;  // 0: pool, 2-D view; 1: pool, decode's view; 2: rows of tokens; 3: pool, groups of rows
    int dtype;
    const void* base;
    int64_t a, b, c, d, e, f;
    bool operator==(const MapKey& o) const {
        return kind == o.kind && dtype == o.dtype && base == o.base && a == o.a && b == o.b && c == o.c &&
               d == o.d && e == o.e && f == o.f;
    }
};
struct MapSlot {
    CUtensorMap map;  // 64-byte aligned type
    MapKey key;
    bool valid;
};
struct MapCache {
    static constexpr int kSlots = 16;
    MapSlot slots[kSlots];
    unsigned next;

    const CUtensorMap* find(const MapKey& key) const {
        for (int i = 0; i < kSlots; ++i)
            if (slots[i].valid && slots[i].key == key) return &slots[i].map;
        return nullptr;
    }
    MapSlot& take() {  // the oldest
        MapSlot& slot = slots[next++ % kSlots];
        slot.valid = false;
        return slot;
    }
};
thread_local MapCache t_pool_maps;
thread_local MapCache t_row_maps;

const CUtensorMap* pool_map(const void* base, int dtype, const pa::PoolShape& shape, bool interleave) {
    const MapKey key{interleave ? 1 : 0, dtype, base, shape.num_blocks, shape.num_kv_heads, shape.block_size,
                     shape.head_dim, 0, 0};
    if (const CUtensorMap* m = t_pool_maps.find(key)) return m;
    MapSlot& slot = t_pool_maps.take();
    if (!encode_pool_map(&slot.map, base, dtype, shape, interleave)) return nullptr;
    slot.key = key;
    slot.valid = true;
    return &slot.map;
}

const CUtensorMap* group_map(const void* base, int dtype, const pa::PoolShape& shape) {
    const MapKey key{3, dtype, base, shape.num_blocks, shape.num_kv_heads, shape.block_size, shape.head_dim, 0, 0};
    if (const CUtensorMap* m = t_pool_maps.find(key)) return m;
    MapSlot& slot = t_pool_maps.take();
    if (!encode_group_map(&slot.map, base, dtype, shape)) return nullptr;
    slot.key = key;
    slot.valid = true;
    return &slot.map;
}

const CUtensorMap* rows_map(const void* base, int dtype, int num_tokens, int num_heads, int head_dim,
                            int64_t token_stride, int box_heads, int box_tokens) {
    const MapKey key{2, dtype, base, num_tokens, num_heads, head_dim, token_stride, box_heads, box_tokens};
    if (const CUtensorMap* m = t_row_maps.find(key)) return m;
    MapSlot& slot = t_row_maps.take();
    if (!encode_rows_map(&slot.map, base, dtype, num_tokens, num_heads, head_dim, token_stride, box_heads, box_tokens))
        return nullptr;
    slot.key = key;
    slot.valid = true;
    return &slot.map;
}

int status_of(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    if (e == cudaErrorNotSupported) return PA_ERR_UNSUPPORTED;
    return PA_ERR_CUDA;
}

constexpr int kAutoPartitionSmall = 256;
constexpr int kAutoPartition = 512;

}  // namespace

namespace pa {

int decode_partition(int64_t num_seqs, int num_kv_heads, int max_context_len, int partition_size) {
    if (partition_size != 0) return partition_size;
    const int dev = current_device();
    const int sms = dev < 0 ? 0 : sm_count(dev);
    if (sms <= 0) return -1;
    // Enough independent (sequence, KV head, partition) items to keep every
    // SM busy through the tail; shorter partitions when the batch is small.
    const int64_t units = num_seqs * num_kv_heads;
    return units * max_parts_for(max_context_len, kAutoPartition) < 4LL * sms ? kAutoPartitionSmall
                                                                             : kAutoPartition;
}

size_t decode_workspace_bytes(int num_seqs, int num_heads, int max_context_len, int partition, int head_dim) {
    return decode_workspace_layout(num_seqs, num_heads, max_parts_for(max_context_len, partition), head_dim).total;
}

namespace host {
int elem_bytes(int dtype) { return ::elem_bytes(dtype); }
bool aligned(const void* p, uintptr_t a) { return ::aligned(p, a); }
int check_cache(const pa_cache_desc* c, PoolShape* shape) { return ::check_cache(c, shape); }
int current_device() { return ::current_device(); }
int* error_word(int dev) { return ::error_word(dev); }
int sm_count(int dev) { return ::sm_count(dev); }
int option(int id) { return ::option(id); }
unsigned long long wait_limit_ns() { return ::wait_limit_ns(); }
int status_of(cudaError_t e) { return ::status_of(e); }
const CUtensorMap* rows_map(const void* base, int dtype, int num_tokens, int num_heads, int head_dim,
                            int64_t token_stride, int box_heads, int box_tokens) {
    return ::rows_map(base, dtype, num_tokens, num_heads, head_dim, token_stride, box_heads, box_tokens);
}
const CUtensorMap* group_map(const void* base, int dtype, const PoolShape& shape) {
    return ::group_map(base, dtype, shape);
}
}  // namespace host

}  // namespace pa

extern "C" {

int pa_abi_version(void) { return PA_ABI_VERSION; }

int pa_set_option(int opt, int value) {
    if (opt < 0 || opt >= kNumOptions || (value != 0 && value != 1)) return PA_ERR_INVALID_ARG;
    option(opt);  // the environment's value first, so that it never overrides this one
    return g_option[opt].exchange(value);
}

int pa_get_option(int opt) {
    if (opt < 0 || opt >= kNumOptions) return PA_ERR_INVALID_ARG;
    return option(opt);
}

const char* pa_status_string(int status) {
    switch (status) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
        case PA_ERR_DEVICE_FAULT: return "PA_ERR_DEVICE_FAULT";
        case PA_ERR_DEVICE_TIMEOUT: return "PA_ERR_DEVICE_TIMEOUT";
        default: return "PA_ERR_UNKNOWN";
    }
}

int pa_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                         const int64_t* slot_mapping, int64_t num_tokens, const pa_cache_desc* cache,
                         void* stream) {
    NvtxRange range("pa_reshape_and_cache");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slot_mapping, 8))
        return PA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    if (option(PA_OPT_DEBUG_CHECKS)) {
        rc = status_of(pa::launch_check_unique_slots(slot_mapping, num_tokens, err, static_cast<cudaStream_t>(stream)));
        if (rc != PA_OK) return rc;
    }
    return status_of(pa::launch_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, num_tokens, shape,
                                                  err, static_cast<cudaStream_t>(stream)));
}

int pa_rotary_and_cache(void* query_out, int64_t query_out_stride, void* key_out, int64_t key_out_stride,
                        const void* query, int64_t query_stride, const void* key, int64_t key_stride,
                        const void* value, int64_t value_stride, const int32_t* positions, const float* cos_sin,
                        int32_t num_positions, int32_t rotary_dim, int32_t interleaved, void* k_cache, void* v_cache,
                        const int64_t* slot_mapping, int64_t num_tokens, int32_t num_heads,
                        const pa_cache_desc* cache, void* stream) {
    NvtxRange range("pa_rotary_and_cache");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0 || num_heads <= 0 || num_heads % shape.num_kv_heads != 0 || num_positions <= 0 ||
        rotary_dim <= 0 || rotary_dim > shape.head_dim || rotary_dim % 2 != 0 || (interleaved != 0 && interleaved != 1))
        return PA_ERR_INVALID_ARG;
    const int64_t q_row = (int64_t)num_heads * shape.head_dim, kv_row = (int64_t)shape.num_kv_heads * shape.head_dim;
    const int per_chunk = 16 / shape.elem_bytes;
    if (query_stride < q_row || query_out_stride < q_row || key_stride < kv_row || value_stride < kv_row ||
        (key_out && key_out_stride < kv_row) || query_stride % per_chunk || query_out_stride % per_chunk ||
        key_stride % per_chunk || value_stride % per_chunk || (key_out && key_out_stride % per_chunk))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!aligned(query_out, 16) || (key_out && !aligned(key_out, 16)) || !aligned(query, 16) || !aligned(key, 16) ||
        !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cos_sin, 16) ||
        !aligned(positions, 4) || !aligned(slot_mapping, 8))
        return PA_ERR_INVALID_ARG;
    // A row that is written where another is still to be read: only whole arrays in place.
    if ((query_out == query && query_out_stride != query_stride) ||
        (key_out && key_out == key && key_out_stride != key_stride))
        return PA_ERR_INVALID_ARG;
    if (!pa::rotary_supported(shape.head_dim, rotary_dim, shape.elem_bytes)) return PA_ERR_UNSUPPORTED;

    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    if (option(PA_OPT_DEBUG_CHECKS)) {
        rc = status_of(pa::launch_check_unique_slots(slot_mapping, num_tokens, err, static_cast<cudaStream_t>(stream)));
        if (rc != PA_OK) return rc;
    }
    pa::RotaryParams p{};
    p.query = query;
    p.key = key;
    p.value = value;
    p.query_out = query_out;
    p.key_out = key_out;
    p.query_stride = query_stride;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.query_out_stride = query_out_stride;
    p.key_out_stride = key_out_stride;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.cos_sin = cos_sin;
    p.num_positions = num_positions;
    p.rotary_dim = rotary_dim;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.num_heads = num_heads;
    p.num_kv_heads = shape.num_kv_heads;
    p.block_size = shape.block_size;
    p.num_slots = shape.num_blocks * shape.block_size;
    p.err = err;
    return status_of(pa::launch_rotary(p, cache->dtype, shape.head_dim, shape.elem_bytes, interleaved != 0, num_tokens,
                                       static_cast<cudaStream_t>(stream)));
}

int pa_plan_step(const int32_t* new_lens, const int32_t* context_lens, int32_t* context_lens_out, int32_t num_seqs,
                 int32_t* free_ring, int32_t ring_size, const int32_t* free_state, int32_t* free_state_out,
                 int64_t num_blocks, int32_t block_size, int32_t* block_tables, int32_t max_blocks_per_seq,
                 int32_t* query_start_loc, int64_t* slot_mapping, int32_t* positions, int32_t max_tokens,
                 void* stream) {
    NvtxRange range("pa_plan_step");
    if (num_seqs < 0 || ring_size <= 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
        max_tokens < 0)
        return PA_ERR_INVALID_ARG;
    if (!aligned(query_start_loc, 4) || !aligned(free_ring, 4) || !aligned(free_state, 4) || !aligned(free_state_out, 4))
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!aligned(new_lens, 4) || !aligned(context_lens, 4) || !aligned(context_lens_out, 4) ||
                         !aligned(block_tables, 4)))
        return PA_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!aligned(slot_mapping, 8) || !aligned(positions, 4))) return PA_ERR_INVALID_ARG;
    if (num_seqs > pa::kMaxStepSeqs || max_tokens >= pa::kMaxStepCount || ring_size >= pa::kMaxStepCount)
        return PA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    pa::StepPlanParams p{};
    p.new_lens = new_lens;
    p.context_lens = context_lens;
    p.context_lens_out = context_lens_out;
    p.num_seqs = num_seqs;
    p.free_ring = free_ring;
    p.ring_size = ring_size;
    p.free_state = free_state;
    p.free_state_out = free_state_out;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.block_tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
    p.ctx_cap = (int)(cap < 0x7fffffffLL ? cap : 0x7fffffffLL);
    p.query_start_loc = query_start_loc;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.max_tokens = max_tokens;
    p.err = err;
    return status_of(pa::launch_step_plan(p, static_cast<cudaStream_t>(stream)));
}

size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t max_context_len,
                                int32_t partition_size, int32_t head_dim) {
    if (num_seqs < 0 || num_heads <= 0 || max_context_len < 0 || head_dim <= 0 || !partition_ok(partition_size))
        return 0;
    const int part = partition_size ? partition_size : kAutoPartitionSmall;
    return pa::decode_workspace_layout(num_seqs, num_heads, max_parts_for(max_context_len, part), head_dim).total;
}

int pa_decode(void* out, int32_t out_dtype, const void* query, const void* k_cache, const void* v_cache,
              const pa_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
              const int32_t* context_lens, int32_t num_seqs, int32_t max_context_len, int32_t num_heads,
              int32_t num_kv_heads, float scale, int32_t partition_size, void* workspace,
              size_t workspace_bytes, void* stream) {
    NvtxRange range("pa_decode");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (elem_bytes(out_dtype) == 0) return PA_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads != cache->num_kv_heads || num_heads % num_kv_heads != 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || !std::isfinite(scale) || !partition_ok(partition_size))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!aligned(out, 16) || !aligned(query, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (!(group == 1 || group == 2 || group == 4 || group == 8)) return PA_ERR_UNSUPPORTED;
    if (!(shape.head_dim == 64 || shape.head_dim == 128)) return PA_ERR_UNSUPPORTED;
    if (!(shape.block_size == 8 || shape.block_size == 16 || shape.block_size == 32)) return PA_ERR_UNSUPPORTED;

    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;

    const int part = pa::decode_partition(num_seqs, num_kv_heads, max_context_len, partition_size);
    if (part <= 0) return PA_ERR_CUDA;
    const int max_parts = max_parts_for(max_context_len, part);
    const pa::DecodeWorkspaceLayout lay = pa::decode_workspace_layout(num_seqs, num_heads, max_parts, shape.head_dim);
    if (!aligned(workspace, 256) || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
    const int64_t items_ub = (int64_t)num_seqs * max_parts * num_kv_heads;
    if (items_ub > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;

    char* ws = static_cast<char*>(workspace);
    pa::DecodeParams p{};
    p.out = out;
    p.out_dtype = out_dtype;
    p.query = query;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = shape.num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.partition_size = part;
    p.max_parts = max_parts;
    const int64_t table_cap = (int64_t)max_blocks_per_seq * shape.block_size;
    const int64_t part_cap = (int64_t)max_parts * part;
    const int64_t cap = table_cap < part_cap ? table_cap : part_cap;
    p.ctx_cap = (int)(cap < 0x7fffffffLL ? cap : 0x7fffffffLL);
    p.next_item = reinterpret_cast<int*>(ws + lay.next_item);
    p.num_items = reinterpret_cast<int*>(ws + lay.num_items);
    p.items = reinterpret_cast<int2*>(ws + lay.items);
    p.num_multi = reinterpret_cast<int*>(ws + lay.num_multi);
    p.multi_seqs = reinterpret_cast<int2*>(ws + lay.multi_seqs);
    p.part_ml = reinterpret_cast<float*>(ws + lay.part_ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.part_o);
    p.err = err;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_flags = option(PA_OPT_DROP_FIRST_FILL) ? pa::kDebugDropFirstFill : 0;
    // Every context fits one partition: no planning kernel, items are implicit.
    p.direct_items = max_parts == 1 ? (int)items_ub : 0;

    if (option(PA_OPT_DEBUG_CHECKS)) {
        rc = status_of(pa::launch_check_decode_inputs(context_lens, block_tables, num_seqs, max_blocks_per_seq,
                                                      shape.block_size, max_context_len, shape.num_blocks, err,
                                                      static_cast<cudaStream_t>(stream)));
        if (rc != PA_OK) return rc;
    }

    pa::DecodeVariant variant = option(PA_OPT_DECODE_KERNEL) ? pa::kDecodeSimt : pa::kDecodeMma;
    const CUtensorMap* tmap_k = nullptr;
    const CUtensorMap* tmap_v = nullptr;
    CUtensorMap k_map, v_map;  // copies: a second lookup may reuse the first one's cache slot
    if (cache->dtype != PA_F32 && variant == pa::kDecodeMma) {
        tmap_k = pool_map(k_cache, cache->dtype, shape, true);
        if (tmap_k) {
            k_map = *tmap_k;
            tmap_v = pool_map(v_cache, cache->dtype, shape, true);
        }
        if (tmap_v) v_map = *tmap_v;
    }
    if (!tmap_k || !tmap_v) variant = pa::kDecodeSimt;
    return status_of(pa::launch_decode(p, cache->dtype, shape.head_dim, shape.block_size, group, (int)items_ub,
                                       variant, &k_map, &v_map, static_cast<cudaStream_t>(stream)));
}

int pa_prefill(void* out, int32_t out_dtype, const void* query, const int32_t* query_start_loc,
               int32_t num_query_tokens, int32_t max_query_len, const void* k_cache, const void* v_cache,
               const pa_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
               const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, float scale,
               void* stream) {
    NvtxRange range("pa_prefill");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (elem_bytes(out_dtype) == 0) return PA_ERR_INVALID_ARG;
    if (num_seqs < 0 || num_query_tokens < 0 || max_query_len < 0 || num_heads <= 0 ||
        num_kv_heads != cache->num_kv_heads || num_heads % num_kv_heads != 0 || max_blocks_per_seq <= 0 ||
        !std::isfinite(scale) || !(scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_query_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!aligned(out, 16) || !aligned(query, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (!(group == 1 || group == 2 || group == 4 || group == 8)) return PA_ERR_UNSUPPORTED;
    if (cache->dtype == PA_F32) return PA_ERR_UNSUPPORTED;
    if (!(shape.head_dim == 64 || shape.head_dim == 128)) return PA_ERR_UNSUPPORTED;
    if (!(shape.block_size == 8 || shape.block_size == 16 || shape.block_size == 32)) return PA_ERR_UNSUPPORTED;

    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;

    pa::PrefillParams p{};
    p.out = out;
    p.out_dtype = out_dtype;
    p.query_start = query_start_loc;
    p.block_tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_query_tokens;
    p.max_query_len = max_query_len;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group_shift = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
    p.block_size = shape.block_size;
    p.num_blocks = shape.num_blocks;
    const int64_t cap = (int64_t)max_blocks_per_seq * shape.block_size;
    p.ctx_cap = (int)(cap < 0x7fffffffLL ? cap : 0x7fffffffLL);
    p.tile_tokens = 128 / group;
    p.tiles_per_seq = (max_query_len + p.tile_tokens - 1) / p.tile_tokens;
    // Pools (K and V) larger than L2: keep each (sequence, KV head)'s query
    // tiles together so that its keys and values are read from HBM once.
    const double pool_bytes = 2.0 * (double)shape.num_blocks * shape.num_kv_heads * shape.block_size *
                              shape.head_dim * shape.elem_bytes;
    p.tiles_adjacent = pool_bytes > (double)l2_bytes(dev) ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    p.wait_limit_ns = wait_limit_ns();

    CUtensorMap tmap_q, tmap_k, tmap_v;  // copies: later lookups may reuse a cache slot
    // One prefill tile: 128 rows (token, grouped head).
    const CUtensorMap* m = rows_map(query, cache->dtype, num_query_tokens, num_heads, shape.head_dim,
                                    (int64_t)num_heads * shape.head_dim, group, 128 / group);
    if (!m) return PA_ERR_UNSUPPORTED;
    tmap_q = *m;
    if (!(m = pool_map(k_cache, cache->dtype, shape, false))) return PA_ERR_UNSUPPORTED;
    tmap_k = *m;
    if (!(m = pool_map(v_cache, cache->dtype, shape, false))) return PA_ERR_UNSUPPORTED;
    tmap_v = *m;
    return status_of(pa::launch_prefill(p, cache->dtype, shape.head_dim, &tmap_q, &tmap_k, &tmap_v,
                                        static_cast<cudaStream_t>(stream)));
}

size_t pa_prompt_attention_workspace_size(int32_t num_seqs, int32_t num_tokens, int32_t num_heads,
                                          int32_t num_kv_heads) {
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        num_heads / num_kv_heads > 128)
        return 0;
    return pa::kPromptHeaderBytes +
           pa::prompt_max_units(num_tokens, num_seqs, 128 / (num_heads / num_kv_heads)) * sizeof(int4);
}

int pa_prompt_attention(void* out, const void* query, int64_t query_stride, const void* key, int64_t key_stride,
                        const void* value, int64_t value_stride, const int32_t* query_start_loc, int32_t num_seqs,
                        int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                        float scale, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange range("pa_prompt_attention");
    if (elem_bytes(dtype) == 0 || num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || head_dim <= 0 || !(scale > 0.f) ||
        !std::isfinite(scale * 1.4426950408889634f))
        return PA_ERR_INVALID_ARG;
    const int64_t q_row = (int64_t)num_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (query_stride < q_row || key_stride < kv_row || value_stride < kv_row || query_stride % head_dim != 0 ||
        key_stride % head_dim != 0 || value_stride % head_dim != 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!aligned(out, 32) || !aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) ||
        !aligned(query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    if (dtype == PA_F32) return PA_ERR_UNSUPPORTED;
    if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
    const int group = num_heads / num_kv_heads;
    if (group > 128) return PA_ERR_UNSUPPORTED;
    constexpr int64_t kMaxStride = (1LL << 39) - 1;  // a tensor copy's strides are below 2^40 bytes
    if (query_stride > kMaxStride || key_stride > kMaxStride || value_stride > kMaxStride) return PA_ERR_UNSUPPORTED;

    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    const int sms = sm_count(dev);
    if (!err || sms <= 0) return PA_ERR_CUDA;

    pa::PromptParams p{};
    p.out = out;
    p.value = value;
    p.value_stride = value_stride;
    p.query_start = query_start_loc;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.tile_tokens = 128 / group;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    p.wait_limit_ns = wait_limit_ns();
    p.debug_flags = option(PA_OPT_DROP_FIRST_FILL) ? pa::kDebugDropFirstFill : 0;
    if (!aligned(workspace, 256) ||
        workspace_bytes < pa_prompt_attention_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads))
        return PA_ERR_WORKSPACE;
    const int64_t units = pa::prompt_max_units(num_tokens, num_seqs, p.tile_tokens);
    if (units * num_kv_heads > 0x40000000LL) return PA_ERR_UNSUPPORTED;  // item numbers stay 32-bit
    if (units * num_kv_heads > sms) {
        // More items than CTAs: a planning kernel lists them.
        char* ws = static_cast<char*>(workspace);
        p.num_units = reinterpret_cast<int*>(ws);
        p.next_item = p.num_units + 1;
        p.items = reinterpret_cast<int4*>(ws + pa::kPromptHeaderBytes);
    }

    CUtensorMap tmap_q, tmap_k, tmap_v;  // copies: later lookups may reuse a cache slot
    const CUtensorMap* m = rows_map(query, dtype, num_tokens, num_heads, head_dim, query_stride, group, p.tile_tokens);
    if (!m) return PA_ERR_UNSUPPORTED;
    tmap_q = *m;
    if (!(m = rows_map(key, dtype, num_tokens, num_kv_heads, head_dim, key_stride, 1, 64))) return PA_ERR_UNSUPPORTED;
    tmap_k = *m;
    if (!(m = rows_map(value, dtype, num_tokens, num_kv_heads, head_dim, value_stride, 1, 64)))
        return PA_ERR_UNSUPPORTED;
    tmap_v = *m;
    return status_of(pa::launch_prompt(p, dtype, head_dim, sms, &tmap_q, &tmap_k, &tmap_v,
                                       static_cast<cudaStream_t>(stream)));
}

int pa_copy_blocks(void* const* k_caches, void* const* v_caches, int32_t num_layers, const int64_t* src_dst_pairs,
                   int64_t num_pairs, const pa_cache_desc* cache, void* stream) {
    NvtxRange range("pa_copy_blocks");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_layers < 1 || num_layers > pa::kMaxCopyLayers || num_pairs < 0 || !k_caches || !v_caches)
        return PA_ERR_INVALID_ARG;
    if (num_pairs == 0) return PA_OK;
    if (!aligned(src_dst_pairs, 8)) return PA_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!aligned(k_caches[l], 16) || !aligned(v_caches[l], 16)) return PA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    if (option(PA_OPT_DEBUG_CHECKS)) {
        rc = status_of(pa::launch_check_pairs(src_dst_pairs, num_pairs, true, err, static_cast<cudaStream_t>(stream)));
        if (rc != PA_OK) return rc;
    }
    return status_of(pa::launch_copy_blocks(k_caches, v_caches, num_layers, src_dst_pairs, num_pairs, shape, err,
                                            static_cast<cudaStream_t>(stream)));
}

namespace {
// Pool memory the GPU can address: device memory, page-locked host memory
// or managed memory -- not pageable host memory.
bool gpu_addressable(const void* p) {
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();  // a failed query leaves no error behind for later calls
        return false;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeHost || a.type == cudaMemoryTypeManaged;
}
}  // namespace

int pa_swap_blocks(void* const* src_k, void* const* src_v, int64_t src_num_blocks, void* const* dst_k,
                   void* const* dst_v, int64_t dst_num_blocks, int32_t num_layers, const int64_t* src_dst_pairs,
                   int64_t num_pairs, const pa_cache_desc* cache, void* stream) {
    NvtxRange range("pa_swap_blocks");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_layers < 1 || num_layers > pa::kMaxCopyLayers || num_pairs < 0 || src_num_blocks <= 0 ||
        dst_num_blocks <= 0 || !src_k || !src_v || !dst_k || !dst_v)
        return PA_ERR_INVALID_ARG;
    if (num_pairs == 0) return PA_OK;
    if (!aligned(src_dst_pairs, 8)) return PA_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!aligned(src_k[l], 16) || !aligned(src_v[l], 16) || !aligned(dst_k[l], 16) || !aligned(dst_v[l], 16))
            return PA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    if (!gpu_addressable(src_dst_pairs)) return PA_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!gpu_addressable(src_k[l]) || !gpu_addressable(src_v[l]) || !gpu_addressable(dst_k[l]) ||
            !gpu_addressable(dst_v[l]))
            return PA_ERR_INVALID_ARG;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    if (option(PA_OPT_DEBUG_CHECKS)) {
        bool same_pool = true;
        for (int l = 0; l < num_layers; ++l)
            if (src_k[l] != dst_k[l] || src_v[l] != dst_v[l]) same_pool = false;
        rc = status_of(pa::launch_check_pairs(src_dst_pairs, num_pairs, same_pool, err,
                                              static_cast<cudaStream_t>(stream)));
        if (rc != PA_OK) return rc;
    }
    return status_of(pa::launch_swap_blocks(src_k, src_v, src_num_blocks, dst_k, dst_v, dst_num_blocks, num_layers,
                                            src_dst_pairs, num_pairs, shape, err, static_cast<cudaStream_t>(stream)));
}

int pa_get_device_error(void* stream, int32_t* code) {
    NvtxRange range("pa_get_device_error");
    if (!code) return PA_ERR_INVALID_ARG;
    *code = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ERR_CUDA;
    int word = 0;
    if (cudaMemcpyFromSymbol(&word, g_device_error, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
    *code = word;
    if (word == 0) return PA_OK;
    return (word & PA_DEVERR_TIMEOUT) ? PA_ERR_DEVICE_TIMEOUT : PA_ERR_DEVICE_FAULT;
}

}  // extern "C"
