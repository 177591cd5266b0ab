// The context object behind the opaque skv_ctx handle (internal; not ABI).
#pragma once

#include <vector>

#include <cuda.h>

#include "skv.h"
#include "skv_internal.cuh"

struct skv_ctx {
    skv_config cfg{};
    skv::Dev d{};
    uint8_t* pool_host = nullptr;  // same memory as d.pool (mapped)
    std::vector<uint8_t> active_h;  // host mirror of the request table
    int32_t* st_req = nullptr;      // staging for skv_assemble_host
    int32_t* st_topk = nullptr;
    int32_t* st_slots = nullptr;
    int32_t* st_hits = nullptr;
    int32_t* st_misses = nullptr;
    uint32_t* host_word = nullptr;  // pinned word for reading the error bits
    cudaEvent_t ev_before = nullptr, ev_after = nullptr;
    int gather_grid = 0;
    CUtensorMap hot_map{};  // TMA view of the hot buffer for the attention consumer (built on first use)
    bool hot_map_ready = false;
    float* q4_scratch = nullptr;  // partial results of skv_attend_q4 (contexts of packed rows only)
    int attend_sms = 0;     // SMs the attention kernel may occupy (0: all)
    int device_sms = 0;     // SMs of the context's device
    int prefix_clusters = 0;  // clusters of skv_attend_prefix that fit on it at once
    int pool_node_wanted = -1;   // host NUMA node the pool was asked to live on (-1: none)
    int pool_node_seen = -1;     // node holding most sampled pool pages (-1: not reported)
    float pool_node_frac = 0.0f; // share of the sampled pages on pool_node_seen
};

namespace skv {
// Sets the message returned by skv_last_cuda_error on this thread.
void set_last_error_message(const char* msg);
// Launches a kernel that may start while the kernel before it on the stream
// still runs (programmatic dependent launch): it executes griddepcontrol.wait
// in every CTA before it reads or writes global memory (its inputs through
// behind_wait, so that the compiler keeps to it), and lets the next such
// kernel start early in turn.  Hides the launch and the kernel's set-up where
// calls follow one another; no kernel waits for one that has not started.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
// The driver's cuTensorMapEncodeTiled, reached through the runtime's entry
// point query (no link against the driver library).
using TensorMapEncoder = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t tensor_map_encoder(TensorMapEncoder* encode);
// Selection of Top-k tokens by index scores (skv_select.cu).  select_stride: scores a unit has room for.
int64_t select_stride(int64_t max_context, int block);
cudaError_t prepare_select();  // once per context, on its device
cudaError_t launch_select(const Dev& d, const skv_index& ix, const int32_t* req_ids, int B, const void* q, const float* w,
                          int32_t* topk, void* workspace, int device_sms, cudaStream_t st, bool withhold_keys = false);
// Kernels around a shared prefix (skv_prefix.cu): once per context, on its device.
cudaError_t prepare_prefix(int* clusters);  // *clusters: those of skv_attend_prefix that are on the chip at once
// Loads skv_assemble_noalloc's static work list on `device` (current) and
// caches its address, so that no later call loads or allocates anything.
cudaError_t noalloc_prepare(int device);
}  // namespace skv
