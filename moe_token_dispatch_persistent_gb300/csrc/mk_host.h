// mk_host.h -- host services shared by the entry points' translation units:
// the device check, the per-(device, stream) workspace caches, tensor maps
// and the device error word.  Defined in mk_api.cu and mk_kernels.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <memory>
#include <mutex>

#include "mk.h"

namespace mk {

// The device error word that mk_get_status() reads and clears.
struct DevError {
    uint32_t code, site, cta, info;
};

// Its address on the current device.
cudaError_t error_word(DevError** out);

// The current device: its id, SM count and error word, or why it cannot be
// used.  The first call on a device sets every kernel's attributes.
mk_status_t host_device(int* dev, int* sms, DevError** err);

// Kernel attributes of the units below, set once per device.
cudaError_t attn_kernel_attributes();  // mk_attn4.cu's too
cudaError_t attn4_kernel_attributes();
cudaError_t ffn_kernel_attributes();

// Workspace caches, one per operator family: their control blocks differ.
enum WsKind { WS_DISPATCH = 0, WS_EP = 1, WS_ATTN = 2, WS_FFN = 3, WS_ATTN4 = 4, WS_PAGES = 5, WS_KINDS = 6 };

// The library's workspace of a kind for (device, stream), grown on demand on
// `st`.  Of a new buffer the first `zero_bytes` are zeroed (WS_DISPATCH, WS_PAGES)
// or all of it (the others, whose counters move with the sizes).  The object holds
// the buffer: keep it until the call's work is enqueued, so that no other thread's
// call frees what this one is about to use.  A call under stream capture gets
// what an earlier call on the stream left, which is then the captured calls'
// alone; without that, memory of the graph (WS_DISPATCH, WS_EP) or
// MK_ERR_WORKSPACE (the others).
struct WsEntry;
class Workspace {
  public:
    Workspace() = default;
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    ~Workspace();
    mk_status_t get(WsKind kind, int dev, cudaStream_t st, size_t need, size_t zero_bytes);
    uint8_t* data() const { return ptr_; }

  private:
    std::shared_ptr<WsEntry> entry_;
    std::unique_lock<std::mutex> lock_;  // of the entry
    uint8_t* ptr_ = nullptr;
    void* own_ = nullptr;                // memory of the graph that the call is captured in
    cudaStream_t stream_ = nullptr;
};

// A 2-D tensor map in the 128-byte swizzle (out-of-range reads give zeros).
CUresult host_encode_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
                        uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer);

inline bool host_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace mk
