// layer_scratch.cu: workspaces of the 16-bit layer operators.
#include "layer16.cuh"

#include <algorithm>
#include <mutex>
#include <vector>

namespace sg {
namespace {

struct Entry {
    int dev;
    cudaStream_t stream;
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
    std::lock_guard<std::mutex> lock(g_mutex);
    Entry *e = nullptr;
    for (auto &w : g_entries)
        if (w.dev == dev && w.stream == stream && w.use == use) e = &w;
    if (!e) {
        g_entries.push_back({dev, stream, use, nullptr, 0});
        e = &g_entries.back();
    }
    if (e->bytes < bytes || e->distrusted) {
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        err = cudaStreamIsCapturing(stream, &capture);
        if (err == cudaSuccess && capture != cudaStreamCaptureStatusNone) err = cudaErrorStreamCaptureUnsupported;
        if (err != cudaSuccess) {
            cudaGetLastError();
            *detail = "a captured call needs a larger or cleared workspace (make a call of its kind and sizes on "
                      "the stream before the capture)";
            return err;
        }
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
    for (auto &w : g_entries) release(w.dev, w.ptr);
    for (auto &w : g_outgrown) release(w.dev, w.ptr);
    cudaSetDevice(cur);
    g_entries.clear();
    g_outgrown.clear();
    return first;
}

}  // namespace sg
