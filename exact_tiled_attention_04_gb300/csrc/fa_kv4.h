// Declarations shared by the host entry points of the 4-bit key/value cache
// (fa_kv4_api.cu) and its kernels.  Not part of the public C ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "fa_host.h"
#include "fa_internal.h"

namespace fa {

// A cache as the kernels see it (fa_kv4_cache_t in 32-bit sizes).
struct Kv4Cache {
    uint8_t* codes[2];   // keys, values: [B * H_kv, capacity, d / 2]
    uint8_t* scales[2];  // [B * H_kv, capacity, d / 16]
    float* weight;       // [B * H_kv, capacity] or nullptr
    int32_t* pos;        // [B * H_kv, capacity] or nullptr
    int32_t* counts;     // [2, B]: length, tokens appended
    int B, H_kv, capacity, d;
};

// The kernels of this file are launched with programmatic serialization: a
// kernel is set up while the one before it in the stream runs, and waits for
// that one's end (and through it for everything earlier) before it touches
// memory that another kernel may have written.
#ifdef __CUDACC__
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream be set up.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif
// Lets a kernel have `smem` bytes of dynamic shared memory, once per device
// and context (a device reset loses the limit).  `done`: per device the context
// that has it; the kernel's own, as is its limit, which every call sets alike.
struct SmemAllowed {
    std::atomic<unsigned long long> ctx_id[host::kMaxCachedDevices] = {};
};
inline cudaError_t allow_smem(const void* kernel, int smem, SmemAllowed& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev < host::kMaxCachedDevices;
    const unsigned long long ctx = host::current_context_id();
    if (cached && ctx != 0 && done.ctx_id[dev].load(std::memory_order_relaxed) == ctx) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // the call made a context current if none was
    if (e == cudaSuccess && cached) done.ctx_id[dev].store(host::current_context_id(), std::memory_order_relaxed);
    return e;
}
// The same for a kernel whose warps move registers among them (setmaxnreg): it
// has to have been compiled for exactly `regs` a thread, as an increase without
// the registers behind it would never return.
inline cudaError_t allow_smem_regs(const void* kernel, int smem, int regs, SmemAllowed& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long ctx = host::current_context_id();
    if (dev < host::kMaxCachedDevices && ctx != 0 && done.ctx_id[dev].load(std::memory_order_relaxed) == ctx)
        return cudaSuccess;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != regs) return cudaErrorInvalidConfiguration;
    return allow_smem(kernel, smem, done);
}
template <class Kernel, class... Args>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Kv4AppendParams {
    Kv4Cache c;
    const void* x[2];     // k, v: [B * H_kv, n, d]
    int32_t* counts_out;  // [2, B]
    DevStatus* status;
    long long n;
    int f16;
};
cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t stream);

struct Kv4ReadParams {
    Kv4Cache c;
    const int32_t* first;  // [B] or nullptr
    void* x[2];            // k, v: [B * H_kv, count, d] or nullptr
    long long count;
    int f16;
};
cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t stream);

struct Kv4EvictParams {
    Kv4Cache from, to;    // to.codes[0] == from.codes[0]: in place
    const float* rank_by;
    int32_t* src;         // [B * H_kv, keep]
    int32_t* counts_out;  // [2, B]
    int keep, sinks;
    int recent;
};
constexpr int kKv4EvictMaxCapacity = 393216;
// Copies into another cache: blocks per head, of kKv4CopyRows slots each.  No
// more entries are kept than the first cache has slots, however large `keep`.
constexpr int kKv4CopyRows = 256;
constexpr int kv4_kept_at_most(int64_t keep, int64_t capacity) {
    return static_cast<int>(keep < capacity ? keep : capacity);
}
constexpr int kv4_copy_blocks(int64_t keep, int64_t capacity) {  // capacity <= kKv4EvictMaxCapacity
    return (kv4_kept_at_most(keep, capacity) + kKv4CopyRows - 1) / kKv4CopyRows;
}
cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream);

// Attention over the cache.  Rows: the R = N_q * group query rows of a
// key/value head, row r = g * N_q + i (query head g of the group, query i),
// in blocks of `rows_per_block`.  A unit is one (sequence, key/value head,
// row block); its keys are cut into slabs of 32, and the slabs of all units,
// in order, into runs of equal length, one per CTA.
struct Kv4FwdParams {
    Kv4Cache c;
    const void* q;        // [B, H, N_q, d]
    void* o;              // [B, H, N_q, d]
    float* lse;           // [B, H, N_q] or nullptr
    const float* weight_in;
    float* weight_out;    // or nullptr
    DevStatus* status;
    unsigned int gen;
    int Nq, group, rows, row_blocks;
    int causal, f16;
    float scale_log2;
    int ctas;             // CTAs of the main kernel
    int single;           // 1: one per unit
    int unit_cost;        // slabs counted for ending a unit
    int join_warps;       // of the second kernel, per row: one or a block
    // workspace
    float* row_lse2;      // [B * H_kv * rows]: base-2 lse of the rows of units that one CTA finished
    float4* part_ml;      // [ctas, 2, rows_per_block]: reference, exact sum, rounded sum
    float* part_o;        // [ctas, 2, rows_per_block, d]
    float* logits;        // [B * H_kv, capacity, rows] scaled, base 2, or nullptr
};
constexpr int kKv4UnitCost = 8;  // slabs that ending a unit costs
int kv4_rows_per_block(int64_t rows);
struct Kv4Plan {
    int ctas = 0;
    bool single = false;
    int unit_cost = 0;
    int join_warps = 1;
};
Kv4Plan kv4_plan(int64_t B, int64_t H_kv, int64_t rows, int64_t capacity, int sms);
cudaError_t launch_kv4_fwd(const Kv4FwdParams& p, cudaStream_t stream);

struct WeightsParams {
    const float* lse;        // [B, H, N_q]
    const float* weight_in;  // or nullptr
    float* weight_out;
    long long weight_stride;
    DevStatus* status;
    unsigned int gen;
    int Nq, Nkv, H, H_kv, group, first_query;
    int causal, causal_offset;
    float scale_log2;
    int splits;              // CTAs (one cluster) that share the query rows of a key block
};
cudaError_t launch_weights(int d, bool f16, const CUtensorMap& q, const CUtensorMap& k, const WeightsParams& p,
                           unsigned int grid, cudaStream_t stream);

}  // namespace fa
