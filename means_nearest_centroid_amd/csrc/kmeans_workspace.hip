// kmeans_workspace.hip -- the memory that the library keeps per stream between
// calls: one scratch buffer and the persistent path's tile queue.
//
// Calls may be captured into a graph, whose replays go on using the addresses
// they were given.  So a buffer that a captured call took is not freed when a
// later call needs a larger one, but kept until kmeans_release_workspace; and
// memory taken during a capture is ordinary memory (hipMalloc), not an
// allocation node of the graph, which later calls could not use.
#include <functional>
#include <map>
#include <mutex>
#include <new>
#include <thread>
#include <tuple>
#include <utility>
#include <vector>

#include "kmeans_internal.h"

namespace kmeans {

namespace {
struct Buffer {
    void *ptr = nullptr;
    size_t bytes = 0;
    bool captured = false;   // a captured call was given it
    bool ordered = true;     // from hipMallocAsync (else hipMalloc)
};
struct Workspace {
    Buffer now;
    std::vector<Buffer> kept;   // outgrown, but graphs still use them
};
struct Queue {
    Buffer buf;
    bool zero = false;          // its counters were zeroed outside a graph
};
// (device, stream, thread) -> what the stream has.  The thread is part of the
// key only for hipStreamPerThread, one handle that names a different stream in
// every thread.  Never destroyed: at process exit the runtime may be gone
// before static destructors run, and it reclaims device memory itself.
using WsKey = std::tuple<int, uintptr_t, size_t>;
std::mutex g_ws_mutex;
auto *g_ws = new std::map<WsKey, Workspace>();
// The persistent path's tile queue: two int32 counters in a small allocation
// of their own (the workspace above is overwritten by other calls, the queue
// must stay zero between launches).
auto *g_queues = new std::map<WsKey, Queue>();
constexpr size_t kQueueBytes = 256;
constexpr size_t kWorkspaceGranule = size_t(1) << 20;

WsKey ws_key(int dev, hipStream_t stream) {
    const size_t thread = stream == hipStreamPerThread
                              ? std::hash<std::thread::id>()(std::this_thread::get_id())
                              : 0;
    return WsKey{dev, reinterpret_cast<uintptr_t>(stream), thread};
}

// The default stream cannot be captured, and must not be asked while another
// one is.
bool is_capturing(hipStream_t stream) {
    if (stream == nullptr)
        return false;
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &status) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return status == hipStreamCaptureStatusActive;
}

hipError_t take(Buffer &b, size_t bytes, bool capturing, hipStream_t stream) {
    void *p = nullptr;
    hipError_t e;
    if (capturing) {
        hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
        if ((e = hipThreadExchangeStreamCaptureMode(&mode)) != hipSuccess)
            return e;
        e = hipMalloc(&p, bytes);
        const hipError_t back = hipThreadExchangeStreamCaptureMode(&mode);
        if (e == hipSuccess && back != hipSuccess) {
            (void)hipFree(p);
            return back;
        }
    } else {
        e = hipMallocAsync(&p, bytes, stream);
    }
    if (e == hipSuccess && p == nullptr)
        e = hipErrorOutOfMemory;
    if (e == hipSuccess)
        b = {p, bytes, capturing, !capturing};
    return e;
}

hipError_t give(Buffer &b, hipStream_t stream) {
    void *p = b.ptr;
    const bool ordered = b.ordered;
    b = {};
    return p == nullptr ? hipSuccess : ordered ? hipFreeAsync(p, stream) : hipFree(p);
}
}  // namespace

WorkspaceLease::WorkspaceLease(hipStream_t stream, size_t bytes) {
    g_ws_mutex.lock();
    int dev = 0;
    error_ = hipGetDevice(&dev);
    if (error_ != hipSuccess)
        return;
    try {
        Workspace &ws = (*g_ws)[ws_key(dev, stream)];
        const bool capturing = is_capturing(stream);
        if (ws.now.bytes < bytes) {
            if (ws.now.captured || (capturing && ws.now.ptr != nullptr)) {
                ws.kept.push_back(ws.now);
                ws.now = {};
            } else if ((error_ = give(ws.now, stream)) != hipSuccess) {
                return;
            }
            const size_t want =
                (bytes + kWorkspaceGranule - 1) / kWorkspaceGranule * kWorkspaceGranule;
            error_ = take(ws.now, want, capturing, stream);
            if (error_ != hipSuccess)
                return;
        }
        ws.now.captured |= capturing;
        ptr_ = ws.now.ptr;
    } catch (const std::bad_alloc &) {   // must not leave a C entry point, nor the lock held
        error_ = hipErrorOutOfMemory;
    }
}

WorkspaceLease::~WorkspaceLease() { g_ws_mutex.unlock(); }

QueueLease::QueueLease(hipStream_t stream) {
    g_ws_mutex.lock();
    int dev = 0;
    error_ = hipGetDevice(&dev);
    if (error_ != hipSuccess)
        return;
    try {
        Queue &q = (*g_queues)[ws_key(dev, stream)];
        const bool capturing = is_capturing(stream);
        if (q.buf.ptr == nullptr) {
            error_ = take(q.buf, kQueueBytes, capturing, stream);
            if (error_ != hipSuccess)
                return;
        }
        if (!q.zero) {
            // Within a capture this zeroes before every replay, where the
            // counters are zero anyway, but not before a call that comes first.
            error_ = launch_zero_queue(static_cast<int *>(q.buf.ptr), stream);
            if (error_ != hipSuccess)
                return;
            q.zero = !capturing;
        }
        ptr_ = static_cast<int *>(q.buf.ptr);
    } catch (const std::bad_alloc &) {
        error_ = hipErrorOutOfMemory;
    }
}

QueueLease::~QueueLease() { g_ws_mutex.unlock(); }

hipError_t release_workspace(hipStream_t stream) {
    std::lock_guard<std::mutex> lock(g_ws_mutex);
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    const WsKey key = ws_key(dev, stream);
    auto qit = g_queues->find(key);
    if (qit != g_queues->end()) {
        Buffer q = qit->second.buf;
        g_queues->erase(qit);
        if ((e = give(q, stream)) != hipSuccess)
            return e;
    }
    auto it = g_ws->find(key);
    if (it == g_ws->end())
        return hipSuccess;
    Workspace ws = std::move(it->second);
    g_ws->erase(it);
    e = give(ws.now, stream);
    for (Buffer &b : ws.kept) {
        const hipError_t k = give(b, stream);
        if (e == hipSuccess)
            e = k;
    }
    return e;
}

}  // namespace kmeans
