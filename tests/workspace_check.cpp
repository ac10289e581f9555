// The per-stream workspace against a model of the runtime's allocator (the HIP
// functions defined here stand before the library's): what a captured graph
// was given stays allocated, and nothing that belongs to a graph is given to
// later calls.  Prints "ok" or what failed.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include <set>

#include "kmeans_internal.h"

bool fail_new = false;
void *operator new(size_t n) {
    void *p = fail_new ? nullptr : std::malloc(n);
    if (p == nullptr)
        throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

namespace {

struct Block {
    bool graph;       // made by a graph's own allocation node: not there between replays
    bool ordered;     // hipMallocAsync's
    bool freed;
};
std::map<void *, Block> blocks;
std::set<hipStream_t> capturing;
hipStreamCaptureMode mode = hipStreamCaptureModeGlobal;
uintptr_t next_address = 0x100000;
bool fail_allocations = false;
bool broken = false;

void expect(bool ok, const char *what) {
    if (!ok) {
        std::printf("failed: %s\n", what);
        broken = true;
    }
}
hipError_t take(void **p, bool graph, bool ordered) {
    if (fail_allocations)
        return hipErrorOutOfMemory;
    *p = reinterpret_cast<void *>(next_address);
    next_address += 0x100000;
    blocks[*p] = {graph, ordered, false};
    return hipSuccess;
}
hipError_t give(void *p) {
    expect(blocks.count(p) == 1 && !blocks[p].freed, "freed once, and was allocated");
    blocks[p].freed = true;
    return hipSuccess;
}
int live() {
    int n = 0;
    for (const auto &b : blocks)
        n += !b.second.freed;
    return n;
}

}  // namespace

extern "C" {
hipError_t hipGetDevice(int *dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus *status) {
    *status = capturing.count(s) ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipThreadExchangeStreamCaptureMode(hipStreamCaptureMode *m) {
    std::swap(*m, mode);
    return hipSuccess;
}
hipError_t hipMallocAsync(void **p, size_t, hipStream_t s) {
    return take(p, capturing.count(s) > 0, true);
}
hipError_t hipFreeAsync(void *p, hipStream_t s) {
    expect(capturing.count(s) == 0, "no free becomes part of a graph");
    expect(blocks[p].ordered, "hipFreeAsync gets what hipMallocAsync gave");
    return give(p);
}
hipError_t hipMalloc(void **p, size_t) {
    if (!capturing.empty() && mode != hipStreamCaptureModeRelaxed)
        return hipErrorStreamCaptureUnsupported;
    return take(p, false, false);
}
hipError_t hipFree(void *p) {
    expect(capturing.empty(), "hipFree outside captures");
    return give(p);
}
}

int eager_zeros = 0;
namespace kmeans {
hipError_t launch_zero_queue(int *, hipStream_t s) {
    eager_zeros += capturing.count(s) == 0;
    return hipSuccess;
}
}

namespace {

hipStream_t stream(int i) { return reinterpret_cast<hipStream_t>(uintptr_t(0x1000) * (i + 1)); }

void *lease(hipStream_t s, size_t bytes) {
    const kmeans::WorkspaceLease l(s, bytes);
    expect(l.error() == hipSuccess && l.ptr() != nullptr, "a workspace");
    return l.ptr();
}
bool usable(void *p) { return blocks.count(p) && !blocks[p].freed && !blocks[p].graph; }

constexpr size_t kMiB = size_t(1) << 20;

}  // namespace

int main() {
    {   // Eager calls alone: one buffer, which grows in stream order.
        const hipStream_t s = stream(0);
        void *a = lease(s, kMiB);
        expect(lease(s, 100) == a, "a small call takes the same buffer");
        void *b = lease(s, 3 * kMiB);
        expect(b != a && blocks[a].freed && usable(b) && live() == 1, "grown, the old one freed");
        expect(blocks[b].ordered, "in stream order");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "released");
    }
    {   // Captured after a first call: the graph's buffer outlives later growth.
        const hipStream_t s = stream(1);
        void *a = lease(s, kMiB);
        capturing.insert(s);
        expect(lease(s, kMiB) == a, "captured calls take the same buffer");
        capturing.clear();
        void *b = lease(s, 5 * kMiB);
        expect(usable(a) && usable(b) && a != b, "growth keeps the captured buffer");
        void *c = lease(s, 9 * kMiB);
        expect(usable(a) && blocks[b].freed && usable(c), "and frees one that no graph has");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "all released");
    }
    {   // Captured without a call before, and grown within the capture.
        const hipStream_t s = stream(2);
        capturing.insert(s);
        void *a = lease(s, kMiB), *b = lease(s, 2 * kMiB);
        expect(mode == hipStreamCaptureModeGlobal, "the thread's capture mode is put back");
        capturing.clear();
        expect(usable(a) && usable(b), "captured calls get memory of their own");
        void *c = lease(s, kMiB);
        expect(c == b, "which later calls share");
        void *d = lease(s, 7 * kMiB);
        expect(usable(a) && usable(b) && usable(d), "and do not free");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "all released");
    }
    {   // A buffer that cannot grow leaves the stream as it was, or without one.
        const hipStream_t s = stream(3);
        capturing.insert(s);
        void *a = lease(s, kMiB);
        capturing.clear();
        fail_allocations = true;
        {
            const kmeans::WorkspaceLease l(s, 2 * kMiB);
            expect(l.error() == hipErrorOutOfMemory, "the failure is reported");
        }
        fail_allocations = false;
        expect(usable(a), "the captured buffer is still there");
        expect(usable(lease(s, 2 * kMiB)), "a later call gets one");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "all released");
    }
    {   // The tile queue: one allocation, zeroed before the first eager call.
        const hipStream_t s = stream(4);
        capturing.insert(s);
        void *a = kmeans::QueueLease(s).ptr();
        capturing.clear();
        expect(usable(a) && eager_zeros == 0, "a queue of its own");
        expect(kmeans::QueueLease(s).ptr() == a && eager_zeros == 1, "zeroed for eager calls");
        expect(kmeans::QueueLease(s).ptr() == a && eager_zeros == 1, "once");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "released");
    }
    {   // Host memory that runs out is a status too, and leaves no lock held.
        const hipStream_t s = stream(5);
        hipError_t w = hipSuccess, q = hipSuccess;
        try {
            fail_new = true;
            w = kmeans::WorkspaceLease(s, kMiB).error();
            q = kmeans::QueueLease(s).error();
            fail_new = false;
        } catch (const std::bad_alloc &) {
            fail_new = false;
            std::printf("failed: an exception left a lease\n");
            return 1;
        }
        expect(w == hipErrorOutOfMemory && q == hipErrorOutOfMemory, "reported");
        expect(usable(lease(s, kMiB)), "a later call gets a workspace");
        expect(kmeans::release_workspace(s) == hipSuccess && live() == 0, "released");
    }
    if (!broken)
        std::printf("ok\n");
    return broken ? 1 : 0;
}
