// Turns of streams (stream_turn.cuh): a list of those that are taken, threaded through
// the callers' stack frames.
#include "stream_turn.cuh"

#include <condition_variable>
#include <mutex>

namespace pk {
namespace {

std::mutex g_mu;
std::condition_variable g_given_back;
StreamTurn *g_taken = nullptr;
int g_waiting = 0;

}  // namespace

StreamTurn::StreamTurn(int device, const void *stream)
    : device_(device), stream_(reinterpret_cast<uintptr_t>(stream)), next_(nullptr) {
    if (stream_ == 1) stream_ = 0;           // the legacy default stream has two names
    std::unique_lock<std::mutex> lock(g_mu);
    auto taken = [this] {
        for (const StreamTurn *t = g_taken; t; t = t->next_)
            if (t->device_ == device_ && t->stream_ == stream_) return true;
        return false;
    };
    while (taken()) {
        ++g_waiting;
        g_given_back.wait(lock);
        --g_waiting;
    }
    next_ = g_taken;
    g_taken = this;
}

StreamTurn::~StreamTurn() {
    std::lock_guard<std::mutex> lock(g_mu);
    StreamTurn **at = &g_taken;
    while (*at != this) at = &(*at)->next_;
    *at = next_;
    if (g_waiting > 0) g_given_back.notify_all();
}

}  // namespace pk
