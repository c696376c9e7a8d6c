// layer_scratch.cu: workspaces of the 16-bit layer operators.
#include "layer16.cuh"

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
std::mutex g_mutex;
std::vector<Entry> g_entries;

}  // namespace

// A new buffer starts with zeros (the counters kept in some of them rely on it).
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
    if (e->bytes < bytes) {
        if (e->ptr) err = cudaFree(e->ptr);  // waits for work that may still use it
        e->ptr = nullptr;
        e->bytes = 0;
        if (err == cudaSuccess) err = cudaMalloc(&e->ptr, bytes);
        if (err == cudaSuccess) {
            e->bytes = bytes;
            err = cudaMemsetAsync(e->ptr, 0, bytes, stream);
        } else {
            e->ptr = nullptr;
        }
        if (err != cudaSuccess) {
            cudaGetLastError();
            *detail = "layer workspace allocation failed";
            return err;
        }
    }
    if (e->distrusted) {
        err = cudaMemsetAsync(e->ptr, 0, e->bytes, stream);
        if (err != cudaSuccess) {
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
    for (auto &w : g_entries) {
        if (!w.ptr) continue;
        cudaSetDevice(w.dev);
        const cudaError_t err = cudaFree(w.ptr);
        if (err != cudaSuccess && first == cudaSuccess) first = err;
    }
    cudaSetDevice(cur);
    g_entries.clear();
    return first;
}

}  // namespace sg
