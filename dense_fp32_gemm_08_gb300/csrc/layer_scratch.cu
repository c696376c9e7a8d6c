// layer_scratch.cu: workspaces of the 16-bit layer operators.
#include "layer16.cuh"

#include <algorithm>
#include <mutex>
#include <thread>
#include <vector>

namespace sg {
namespace {

// A handle does not identify a stream: cudaStreamPerThread names one of each host thread, and a
// destroyed stream's handle may be given to a new one while the old one's kernels still run. The
// stream's id does, but it cannot be asked for while the stream is being captured. The buffers are
// then the ones that the handle named last, outside a capture.
struct Name {
    int dev;
    cudaStream_t handle;
    std::thread::id thread;  // of cudaStreamPerThread
    bool operator==(const Name &o) const { return dev == o.dev && handle == o.handle && thread == o.thread; }
};
struct Entry {
    Name name;
    bool named = true;  // false: the handle has named another stream since
    unsigned long long stream;  // its id
    int use;
    void *ptr;
    size_t bytes;
    bool distrusted = false;  // to be cleared before its next use
};
// A buffer that became too small. A graph captured while it was in use holds its address, so it lives
// until release_layer_workspaces().
struct Outgrown {
    int dev;
    void *ptr;
};
std::mutex g_mutex;
std::vector<Entry> g_entries;
std::vector<Outgrown> g_outgrown;

}  // namespace

// A new buffer starts with zeros (the counters kept in some of them rely on it). While the stream is
// being captured no buffer is allocated or cleared: the clearing would become part of the graph.
cudaError_t layer_scratch(LayerScratch use, cudaStream_t stream, size_t bytes, void **out,
                          const char **detail) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) {
        *detail = "cudaGetDevice failed";
        return err;
    }
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    err = cudaStreamIsCapturing(stream, &status);
    const bool captured = status != cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (err == cudaSuccess && !captured) err = cudaStreamGetId(stream, &id);
    if (err != cudaSuccess) {
        cudaGetLastError();
        *detail = "the stream cannot be used now";
        return err;
    }
    const Name name{dev, stream, stream == cudaStreamPerThread ? std::this_thread::get_id() : std::thread::id()};
    std::lock_guard<std::mutex> lock(g_mutex);
    Entry *e = nullptr;
    for (auto &w : g_entries)
        if (w.use == use && (captured ? w.named && w.name == name : w.stream == id && w.name.dev == dev)) e = &w;
    if ((!e || e->bytes < bytes || e->distrusted) && captured) {
        *detail = "a captured call needs a larger or cleared workspace (make a call of its kind and sizes on the "
                  "stream before the capture)";
        return cudaErrorStreamCaptureUnsupported;
    }
    if (!e) {
        for (auto &w : g_entries)
            if (w.name == name && w.stream != id) w.named = false;
        Entry fresh{name, true, id, use, nullptr, 0};
        g_entries.push_back(fresh);
        e = &g_entries.back();
    }
    if (e->bytes < bytes) {
        // Half as much again at least, so that the outgrown buffers add up to twice the last one at most.
        g_outgrown.reserve(g_outgrown.size() + 1);
        size_t size = std::max(bytes, e->bytes + e->bytes / 2);
        void *fresh = nullptr;
        err = cudaMalloc(&fresh, size);
        if (err != cudaSuccess && size > bytes) {
            size = bytes;
            err = cudaMalloc(&fresh, size);
        }
        if (err != cudaSuccess) {
            cudaGetLastError();
            *detail = "layer workspace allocation failed";
            return err;
        }
        if (e->ptr) g_outgrown.push_back({dev, e->ptr});
        e->ptr = fresh;
        e->bytes = size;
        e->distrusted = true;
    }
    if (e->distrusted) {
        err = cudaMemsetAsync(e->ptr, 0, e->bytes, stream);
        if (err != cudaSuccess) {
            cudaGetLastError();
            *detail = "layer workspace reset failed";
            return err;
        }
        e->distrusted = false;
    }
    *out = e->ptr;
    return cudaSuccess;
}

void layer_scratch_distrust() {
    std::lock_guard<std::mutex> lock(g_mutex);
    for (auto &w : g_entries) w.distrusted = w.ptr != nullptr;
}

cudaError_t release_layer_workspaces() {
    std::lock_guard<std::mutex> lock(g_mutex);
    cudaError_t first = cudaSuccess;
    int cur = 0;
    cudaGetDevice(&cur);
    auto release = [&](int dev, void *ptr) {
        if (!ptr) return;
        cudaSetDevice(dev);
        const cudaError_t err = cudaFree(ptr);
        if (err != cudaSuccess && first == cudaSuccess) first = err;
    };
    for (auto &w : g_entries) release(w.name.dev, w.ptr);
    for (auto &w : g_outgrown) release(w.dev, w.ptr);
    cudaSetDevice(cur);
    g_entries.clear();
    g_outgrown.clear();
    return first;
}

}  // namespace sg
