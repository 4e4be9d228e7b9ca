// Who holds which tile counter of a handle's expert products (host side).  Two
// launches that may run side by side must not draw from one counter.  A stream's
// launches follow each other, so each stream has one, found by the stream's id
// (ids are not used again, and nothing says when a stream is gone: these are not
// given back).  A captured call has one of its own, because its graph can run
// beside anything; it comes back when the graph, and whatever was instantiated from
// it, is gone and has run.  Graphs are destroyed on any thread and may outlive the
// handle: the book is kept until the last holder lets go.
#pragma once

#include <stdint.h>
#include <stdlib.h>

#include <atomic>
#include <new>

namespace ep {

// Two words each on the device (32 KB per handle).
constexpr int kStreamCounters = 512, kCapturedCounters = 3584;

class TileCounters {
   public:
    // A captured call's counter: what the graph holds on to.
    struct Captured {
        TileCounters *book;
        int index;  // from kStreamCounters on
    };

    static TileCounters *create() { return new (std::nothrow) TileCounters(); }

    // The counter of a stream, -1 when all are taken.  Callers of one handle do not overlap.
    int of_stream(unsigned long long id) {
        for (int i = 0; i < streams_; ++i)
            if (stream_[i] == id) return i;
        if (streams_ == kStreamCounters) return -1;
        stream_[streams_] = id;
        return streams_++;
    }
    // A counter for a captured call, to be given back with `give_back`; nullptr when all are taken.
    Captured *take() {
        Captured *c = static_cast<Captured *>(malloc(sizeof(Captured)));
        if (c == nullptr) return nullptr;
        lock();
        int i = -1;
        if (back_ > 0)
            i = free_[--back_];
        else if (fresh_ < kCapturedCounters)
            i = fresh_++;
        unlock();
        if (i < 0) {
            free(c);
            return nullptr;
        }
        holders_.fetch_add(1, std::memory_order_relaxed);
        c->book = this;
        c->index = kStreamCounters + i;
        return c;
    }
    // Makes no CUDA call: a graph's destructor runs it.
    static void give_back(void *captured) {
        Captured *c = static_cast<Captured *>(captured);
        TileCounters *book = c->book;
        book->lock();
        book->free_[book->back_++] = (uint16_t)(c->index - kStreamCounters);
        book->unlock();
        free(c);
        book->release();
    }
    void release() {
        if (holders_.fetch_sub(1, std::memory_order_acq_rel) == 1) delete this;
    }
    int streams() const { return streams_; }
    int captured() {
        lock();
        const int n = fresh_ - back_;
        unlock();
        return n;
    }

   private:
    TileCounters() = default;
    void lock() {
        while (busy_.test_and_set(std::memory_order_acquire)) {
        }
    }
    void unlock() { busy_.clear(std::memory_order_release); }

    std::atomic<int> holders_{1};
    std::atomic_flag busy_ = ATOMIC_FLAG_INIT;
    int streams_ = 0, fresh_ = 0, back_ = 0;
    unsigned long long stream_[kStreamCounters];
    uint16_t free_[kCapturedCounters];
};

}  // namespace ep
