// The layer operators' workspaces on a fake CUDA runtime: what is allocated, freed and cleared, and
// when. Prints one line per failed expectation; exits with their number.
#include "layer_scratch.cu"

#include <cstdio>
#include <cstdlib>
#include <map>

namespace {
std::map<void *, size_t> live;
size_t room = ~static_cast<size_t>(0);  // of one allocation
int clears = 0, failures = 0, device = 0;
std::map<cudaStream_t, unsigned long long> ids;  // of handles that are not their own id
bool fail_clear = false;
cudaStream_t captured = nullptr;  // the stream that is being captured

void expect(bool ok, const char *what) {
    if (ok) return;
    std::printf("failed: %s\n", what);
    ++failures;
}
void *get(cudaStream_t stream, size_t bytes, sg::LayerScratch use = sg::kScratchPack) {
    void *p = nullptr;
    const char *detail = "";
    return sg::layer_scratch(use, stream, bytes, &p, &detail) == cudaSuccess ? p : nullptr;
}
cudaStream_t stream_at(size_t handle) { return reinterpret_cast<cudaStream_t>(handle); }
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int *d) { return *d = device, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return device = d, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t bytes) {
    if (bytes > room) return cudaErrorMemoryAllocation;
    *p = std::malloc(1);
    live[*p] = bytes;
    return cudaSuccess;
}
cudaError_t cudaFree(void *p) {
    expect(live.erase(p) == 1, "only live buffers are freed");
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *p, int, size_t bytes, cudaStream_t) {
    expect(live.count(p) && bytes <= live[p], "a clear stays inside its buffer");
    if (fail_clear) return cudaErrorUnknown;
    ++clears;
    return cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long *id) {
    expect(s != captured, "the id is not asked for during the stream's capture (which that ends)");
    return *id = ids.count(s) ? ids[s] : reinterpret_cast<size_t>(s), cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t q, cudaStreamCaptureStatus *s) {
    return *s = q == captured ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone, cudaSuccess;
}
}

int main() {
    const cudaStream_t s = stream_at(0x1000), t = stream_at(0x2000);
    void *a = get(s, 1000);
    expect(a && clears == 1, "a new buffer is cleared once");
    expect(get(s, 500) == a && get(s, 1000) == a && clears == 1, "a large enough buffer is used again as it is");
    expect(get(t, 1000) != a && get(s, 1000, sg::kScratchDz) != a, "streams and uses do not share");

    void *mine = get(cudaStreamPerThread, 1000);
    ids[cudaStreamPerThread] = 77;  // the same handle in another host thread
    expect(get(cudaStreamPerThread, 1000) != mine, "each thread's default stream has its own");
    void *old = get(t, 1000);
    ids[t] = 78;  // a stream created after `t` was destroyed may get its handle
    expect(get(t, 1000) != old, "a handle used again is another stream");
    ids.clear();
    expect(get(cudaStreamPerThread, 1000) == mine, "and the first thread's is still there");

    void *b = get(s, 1001);
    expect(b && b != a && live.count(a), "an outgrown buffer, whose address a graph may hold, is kept");
    expect(live[b] >= 1500, "growth is geometric");
    expect(get(s, 1001) == b && get(s, live[b]) == b, "the larger one is used from then on");

    captured = s;
    size_t buffers = live.size();
    int cleared = clears;
    expect(get(s, 1500) == b, "a capture may use what is there");
    expect(!get(s, 1 << 20) && live.size() == buffers && clears == cleared, "a capture does not grow a buffer");
    captured = stream_at(0x3000);
    expect(!get(captured, 16), "a capture allocates none");
    expect(get(s, 16) == b, "another stream goes on meanwhile");
    captured = s;
    sg::layer_scratch_distrust();
    expect(!get(s, 16) && clears == cleared, "a capture does not clear a buffer");
    captured = nullptr;
    expect(get(s, 16) == b && clears == cleared + 1, "the next call outside a capture clears it");
    expect(get(s, 16) == b && clears == cleared + 1, "once");

    const cudaStream_t again = stream_at(0x4000);
    void *first = get(again, 64), *first_dz = get(again, 64, sg::kScratchDz);
    ids[again] = 79;  // destroyed, and its handle given to a new stream
    void *second = get(again, 64);
    captured = again;
    expect(second != first && get(again, 64) == second, "a capture uses the buffers of the handle's latest stream");
    expect(first_dz && !get(again, 64, sg::kScratchDz), "and none of the streams before it");
    captured = nullptr;

    fail_clear = true;
    expect(!get(s, 1 << 16), "a clear that fails fails the call");
    fail_clear = false;
    cleared = clears;
    expect(get(s, 1 << 16) && clears == cleared + 1, "and the buffer is cleared before its first use");

    void *c = get(s, 1 << 20);
    room = (1 << 20) + 1;
    expect(get(s, room) != nullptr, "the exact size when there is no room for more");
    room = 100;
    expect(!get(s, 1 << 22) && live.count(c), "a failed growth frees nothing");
    expect(get(s, 1 << 20) != nullptr, "and leaves the buffer in use");
    room = ~static_cast<size_t>(0);

    expect(sg::release_layer_workspaces() == cudaSuccess && live.empty(), "release frees every buffer");
    expect(get(s, 16) != nullptr, "and the next call starts anew");
    sg::release_layer_workspaces();
    return failures;
}
