// The library's workspace caches without a GPU: mk_api.cu compiled as host code
// against a CUDA runtime that only keeps a log per stream.  Each scenario
// drives public entry points and then checks, in the order of the stream,
// that every launch finds its workspace allocated and nobody else's.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <utility>
#include <vector>

#include "mk.h"
#include "mk_common.h"
#include "mk_host.h"

// ------------------------------------------------------- the fake runtime --

namespace {

enum What { ALLOC, FREE, ZERO, LAUNCH, SYNC, COPY };
struct Op {
    What what;
    uintptr_t ptr;
    cudaStream_t stream;
    bool captured;
};

std::mutex mu;
std::vector<Op> ops;                          // in the order they were enqueued
std::map<uintptr_t, size_t> sizes;
uintptr_t next_ptr = 0x10000000;
std::map<cudaStream_t, bool> capturing;
std::map<cudaStream_t, unsigned long long> ids;  // of handles that do not stand for themselves
bool invalidated = false;                     // a call that a capture does not survive
thread_local unsigned long long per_thread_id = 0;
std::atomic<unsigned long long> threads_seen{1000};
thread_local std::function<void()> on_encode;  // between a call's workspace and its launch

bool is_capturing(cudaStream_t s) {
    auto it = capturing.find(s);
    return it != capturing.end() && it->second;
}
void log(What w, const void* p, cudaStream_t s) {
    ops.push_back({w, reinterpret_cast<uintptr_t>(p), s, is_capturing(s)});
}

CUresult CUDAAPI fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    if (on_encode) {
        auto f = std::move(on_encode);
        on_encode = nullptr;
        f();
    }
    return CUDA_SUCCESS;
}

cudaError_t launched(const void* ws, cudaStream_t st) {
    std::lock_guard<std::mutex> l(mu);
    log(LAUNCH, ws, st);
    return cudaSuccess;
}

}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
    const bool enc = std::strcmp(name, "cuTensorMapEncodeTiled") == 0;
    *fn = enc ? reinterpret_cast<void*>(fake_encode) : nullptr;
    *q = enc ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
    return cudaSuccess;
}
cudaError_t cudaMallocAsync(void** p, size_t n, cudaStream_t s) {
    std::lock_guard<std::mutex> l(mu);
    *p = reinterpret_cast<void*>(next_ptr);
    sizes[next_ptr] = n;
    next_ptr += (n + 0xffff) & ~size_t(0xffff);
    log(ALLOC, *p, s);
    return cudaSuccess;
}
cudaError_t cudaFreeAsync(void* p, cudaStream_t s) {
    std::lock_guard<std::mutex> l(mu);
    log(FREE, p, s);
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int, size_t, cudaStream_t s) {
    std::lock_guard<std::mutex> l(mu);
    log(ZERO, p, s);
    return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
    std::lock_guard<std::mutex> l(mu);
    log(SYNC, nullptr, nullptr);
    log(FREE, p, nullptr);
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
    std::lock_guard<std::mutex> l(mu);
    for (const auto& c : capturing) invalidated = invalidated || c.second;
    log(SYNC, nullptr, nullptr);
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* c) {
    std::lock_guard<std::mutex> l(mu);
    *c = is_capturing(s) ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) {
    std::lock_guard<std::mutex> l(mu);
    if (is_capturing(s)) {  // the capture is lost with this
        invalidated = true;
        return cudaErrorStreamCaptureUnsupported;
    }
    if (s == cudaStreamPerThread) {
        if (!per_thread_id) per_thread_id = ++threads_seen;
        *id = per_thread_id;
    } else if (s == nullptr || s == cudaStreamLegacy) {
        *id = 1;
    } else {
        auto it = ids.find(s);
        *id = it != ids.end() ? it->second : 5000000 + reinterpret_cast<uintptr_t>(s);
    }
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* to, const void* from, size_t, cudaMemcpyKind kind, cudaStream_t s) {
    std::lock_guard<std::mutex> l(mu);
    log(COPY, kind == cudaMemcpyHostToDevice ? to : from, s);
    return cudaSuccess;
}
// what no scenario reaches
cudaError_t cudaMalloc(void**, size_t) { return cudaErrorNotSupported; }
cudaError_t cudaMemset(void*, int, size_t) { return cudaErrorNotSupported; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t*, unsigned) { return cudaErrorNotSupported; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaErrorNotSupported; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t*, unsigned) { return cudaErrorNotSupported; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}

namespace mk {
cudaError_t launch_fused(const Params& p, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                         const CUtensorMap&, int, cudaStream_t st) {
    return launched(p.ctl, st);
}
cudaError_t launch_unfused(const Params& p, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                           const CUtensorMap&, int, cudaStream_t st) {
    return launched(p.ctl, st);
}
cudaError_t launch_ep(const Params& p, const CUtensorMap*, const CUtensorMap&, const CUtensorMap&, int,
                      cudaStream_t st) {
    return launched(p.ep_ctl[0], st);
}
cudaError_t set_kernel_attributes() { return cudaSuccess; }
cudaError_t attn_kernel_attributes() { return cudaSuccess; }
cudaError_t ffn_kernel_attributes() { return cudaSuccess; }
cudaError_t fused_max_blocks_per_sm(int* n) { return *n = 1, cudaSuccess; }
cudaError_t read_and_clear_error(uint32_t out[4], cudaStream_t) { return out[0] = 0, cudaSuccess; }
cudaError_t error_word(DevError** out) { return *out = nullptr, cudaSuccess; }
void noalloc_forget_scratch() {}
}  // namespace mk

// ------------------------------------------------------------- scenarios --

namespace {

int failures = 0;
void expect(bool ok, const char* what) {
    if (!ok) {
        std::printf("FAILED: %s\n", what);
        ++failures;
    }
}

// One dispatch call of T tokens: the larger T, the larger its workspace.
mk_status_t call(cudaStream_t st, int T) {
    void* p = reinterpret_cast<void*>(0x100);
    mk_config_t c;
    mk_config_default(&c);
    c.gather = MK_GATHER_STAGED;
    return mk_moe_dispatch_gemm_ex(p, static_cast<float*>(p), T, 64, 8, 2, p, 64, p, static_cast<int32_t*>(p),
                                   static_cast<int32_t*>(p), static_cast<float*>(p), st, &c, nullptr, 0);
}
// The same through the expert-parallel cache.
mk_status_t call_ep(cudaStream_t st, int T) {
    void* p = reinterpret_cast<void*>(0x100);
    return mk_moe_ep_sim(p, static_cast<float*>(p), T, 64, 8, 2, p, 64, 2, p, static_cast<int32_t*>(p),
                         static_cast<int32_t*>(p), static_cast<float*>(p), nullptr, st, nullptr, nullptr, 0);
}

// Host buffers in and out, through the staging of the stream.
mk_status_t call_host(cudaStream_t st, int T) {
    void* p = reinterpret_cast<void*>(0x100);
    return mk_moe_dispatch_gemm_host(p, static_cast<float*>(p), T, 64, 8, 2, p, 64, p, static_cast<int32_t*>(p),
                                     static_cast<int32_t*>(p), static_cast<float*>(p), st, nullptr);
}

cudaStream_t stream(int i) { return reinterpret_cast<cudaStream_t>(uintptr_t(0x5000 + 16 * i)); }

// The allocation that holds an address.
uintptr_t buffer_of(uintptr_t p) {
    auto it = sizes.upper_bound(p);
    return it == sizes.begin() ? 0 : (--it)->first;
}
// Every launch after its buffer's allocation on the same stream and before its release.
void expect_live() {
    std::map<uintptr_t, bool> live;
    for (const Op& o : ops) {
        if (o.what == ALLOC) live[o.ptr] = true;
        if (o.what == FREE) live[o.ptr] = false;
        if (o.what == LAUNCH) expect(live[buffer_of(o.ptr)], "a launch finds its workspace allocated");
        if (o.what == COPY) expect(live[buffer_of(o.ptr)], "a copy finds its staging allocated");
    }
}
int count(What w) {
    int n = 0;
    for (const Op& o : ops) n += o.what == w;
    return n;
}

// Two threads on one stream; the second needs a larger buffer while the first
// stands between its look-up and its launch.
void growth(mk_status_t (*one)(cudaStream_t, int)) {
    expect(one(stream(0), 64) == MK_OK, "first call");
    std::mutex m;
    std::condition_variable cv;
    bool inside = false, grown = false;
    std::thread a([&] {
        on_encode = [&] {
            std::unique_lock<std::mutex> l(m);
            inside = true;
            cv.notify_all();
            // the other call gets the time to pass this one, if it can
            cv.wait_for(l, std::chrono::milliseconds(500), [&] { return grown; });
        };
        expect(one(stream(0), 64) == MK_OK, "the small call");
    });
    std::thread b([&] {
        {
            std::unique_lock<std::mutex> l(m);
            cv.wait(l, [&] { return inside; });
        }
        expect(one(stream(0), 4096) == MK_OK, "the large call");
        std::lock_guard<std::mutex> l(m);
        grown = true;
        cv.notify_all();
    });
    a.join();
    b.join();
    expect(count(LAUNCH) == 3, "three launches");
    expect(count(FREE) == (one == call_host ? 2 : 1), "the small buffers are given back");
    expect_live();
}

// The buffers are released while another thread stands there.
void release_under_a_call(mk_status_t (*one)(cudaStream_t, int)) {
    std::mutex m;
    std::condition_variable cv;
    bool inside = false, released = false;
    std::thread a([&] {
        on_encode = [&] {
            std::unique_lock<std::mutex> l(m);
            inside = true;
            cv.notify_all();
            cv.wait_for(l, std::chrono::milliseconds(500), [&] { return released; });
        };
        expect(one(stream(0), 64) == MK_OK, "the call");
    });
    std::thread b([&] {
        {
            std::unique_lock<std::mutex> l(m);
            cv.wait(l, [&] { return inside; });
        }
        mk_release_workspace();
        std::lock_guard<std::mutex> l(m);
        released = true;
        cv.notify_all();
    });
    a.join();
    b.join();
    expect(one(stream(0), 64) == MK_OK, "a call afterwards");
    expect_live();
}

// The per-thread default stream is one handle for another stream in each thread.
void per_thread() {
    uintptr_t mine[2] = {0, 0};
    for (int i = 0; i < 2; ++i)
        std::thread([&, i] {
            expect(call(cudaStreamPerThread, 64) == MK_OK, "the call");
            expect(call(cudaStreamPerThread, 64) == MK_OK, "the call again");
            mine[i] = buffer_of(ops.back().ptr);
        }).join();
    expect(mine[0] != mine[1], "two threads' streams have a workspace each");
    expect(count(ALLOC) == 2, "and keep it");
    expect_live();
}

// A stream is destroyed and another gets its handle: the first one's work may
// still be running on the buffer.
void recycled_handle() {
    expect(call(stream(3), 64) == MK_OK, "first stream");
    ids[stream(3)] = 77;
    expect(call(stream(3), 64) == MK_OK, "second stream");
    uintptr_t last = 0;
    bool settled = true;
    for (const Op& o : ops) {
        if (o.what == SYNC) settled = true;
        if (o.what != LAUNCH) continue;
        expect(settled || buffer_of(o.ptr) != last, "work of the old stream has ended before its buffer is used");
        last = buffer_of(o.ptr);
        settled = false;
    }
    const int before = count(SYNC);
    expect(call(stream(3), 64) == MK_OK, "second stream again");
    expect(count(SYNC) == before, "no wait in later calls");
    expect_live();
}

// A captured call takes the buffer of the call before.
void captured_call(cudaStream_t st) {
    expect(call(st, 64) == MK_OK, "call before the capture");
    const uintptr_t first = buffer_of(ops.back().ptr);
    capturing[st] = true;
    expect(call(st, 64) == MK_OK, "a captured call");
    capturing[st] = false;
    expect(buffer_of(ops.back().ptr) == first && ops.back().captured, "on the same buffer");
    expect(!invalidated, "the capture survives");
    expect_live();
}

// What a captured call uses is the graph's: no later call frees it or works in it.
void capture_keeps(mk_status_t (*one)(cudaStream_t, int)) {
    const cudaStream_t st = stream(1);
    auto captured = [&](int T) {
        capturing[st] = true;
        expect(one(st, T) == MK_OK, "a captured call");
        capturing[st] = false;
        return buffer_of(ops.back().ptr);
    };
    expect(one(st, 64) == MK_OK, "call before the capture");
    const uintptr_t graph = captured(64);
    expect(one(st, 64) == MK_OK, "the same call afterwards");
    expect(buffer_of(ops.back().ptr) != graph, "works in another buffer");
    expect(one(st, 4096) == MK_OK, "a larger one");
    const uintptr_t second = captured(4096);
    expect(one(st, 4096) == MK_OK, "the larger one afterwards");
    expect(buffer_of(ops.back().ptr) != second, "works in another buffer");
    expect(captured(64) == second, "smaller calls share what captured calls of the stream have");
    ids[st] = 99;  // another stream with that handle
    expect(one(st, 64) == MK_OK, "the other stream's call");
    for (const Op& o : ops) expect(o.what != FREE || (o.ptr != graph && o.ptr != second), "a graph's buffer stays");
    for (const Op& o : ops) expect(!o.captured || o.what == LAUNCH, "nothing but launches is captured");
    mk_release_workspace();
    int freed = 0;
    for (const Op& o : ops) freed += o.what == FREE && (o.ptr == graph || o.ptr == second);
    expect(freed == 2, "until everything is released");
    expect(!invalidated, "the captures survive");
    expect_live();
}

// Without an earlier call on the stream the memory is the graph's own.
void capture_alone() {
    const cudaStream_t st = stream(2);
    capturing[st] = true;
    expect(call(st, 64) == MK_OK, "a captured call");
    capturing[st] = false;
    expect(ops.size() == 4 && ops[0].what == ALLOC && ops[1].what == ZERO && ops[2].what == LAUNCH &&
               ops[3].what == FREE && ops[3].ptr == ops[0].ptr,
           "allocated, zeroed, used and freed in the graph");
    const uintptr_t graph = ops[0].ptr;
    expect(call(st, 64) == MK_OK, "a call afterwards");
    expect(buffer_of(ops.back().ptr) != graph, "works in another buffer");
    expect_live();
}

// The operators of a decode step refuse that.
void capture_refused() {
    const cudaStream_t st = stream(2);
    auto get = [&](size_t need) {
        mk::Workspace w;
        const mk_status_t s = w.get(mk::WS_FFN, 0, st, need, need);
        expect((s == MK_OK) == (w.data() != nullptr), "a buffer with MK_OK");
        return s;
    };
    capturing[st] = true;
    expect(get(1000) == MK_ERR_WORKSPACE, "no buffer yet");
    capturing[st] = false;
    expect(get(1000) == MK_OK, "a call");
    capturing[st] = true;
    expect(get(1000) == MK_OK, "its buffer");
    expect(get(100000) == MK_ERR_WORKSPACE, "too small");
    for (const Op& o : ops) expect(!o.captured, "nothing is captured");
}

}  // namespace

int main(int argc, char** argv) {
    const std::string name = argc > 1 ? argv[1] : "";
    if (name == "growth") growth(call);
    else if (name == "growth_ep") growth(call_ep);
    else if (name == "growth_host") growth(call_host);
    else if (name == "release") release_under_a_call(call);
    else if (name == "release_host") release_under_a_call(call_host);
    else if (name == "per_thread") per_thread();
    else if (name == "recycled_handle") recycled_handle();
    else if (name == "captured_call") captured_call(stream(4));
    else if (name == "captured_call_per_thread") captured_call(cudaStreamPerThread);
    else if (name == "capture_keeps") capture_keeps(call);
    else if (name == "capture_keeps_ep") capture_keeps(call_ep);
    else if (name == "capture_alone") capture_alone();
    else if (name == "capture_refused") capture_refused();
    else return std::printf("no such scenario\n"), 2;
    std::printf("%s: %zu operations, %d failures\n", name.c_str(), ops.size(), failures);
    return failures ? 1 : 0;
}
