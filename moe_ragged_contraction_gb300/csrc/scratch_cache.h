// Scratch blocks kept per (device, stream). Host logic only: the allocator is a
// parameter, so that it can be tested without a GPU.
#pragma once

#include <stddef.h>

#include <deque>
#include <mutex>
#include <vector>

namespace mxw {

enum class Scratch { ok, capturing, failed };

// Alloc: int allocate(void** p, size_t bytes, Stream s) and int release(void* p,
// Stream s), both in stream order; 0 is success.
template <class Stream, class Alloc>
class ScratchCache {
   public:
    // A block of `need` bytes or more for work on `stream`. Growth releases the old
    // block in stream order and allocates the new one in stream order, so earlier
    // calls on the same stream finish with the old block first. While the stream is
    // being captured into a graph nothing is allocated or released (a captured
    // allocation would belong to the graph): Scratch::capturing where the block is
    // too small. A block that was handed out under capture is never released: the
    // graph holds its address, and nothing tells when the graph is gone. `error`
    // receives the allocator's code with Scratch::failed.
    Scratch get(Alloc& alloc, int dev, Stream stream, size_t need, bool capturing, void** out, int* error) {
        Block* b = find(dev, stream);
        if (b && b->bytes >= need) {
            b->in_graph |= capturing;
            *out = b->ptr;
            return Scratch::ok;
        }
        if (capturing) return Scratch::capturing;
        if (!b) {
            blocks_.push_back(Block{dev, stream, nullptr, 0, false});
            b = &blocks_.back();
        }
        if (b->ptr && !b->in_graph) {
            *error = alloc.release(b->ptr, stream);
            if (*error) return Scratch::failed;
        }
        b->ptr = nullptr;
        b->bytes = 0;
        b->in_graph = false;
        *error = alloc.allocate(&b->ptr, need, stream);
        if (*error) return Scratch::failed;
        b->bytes = need;
        *out = b->ptr;
        return Scratch::ok;
    }

   private:
    struct Block {
        int dev;
        Stream stream;
        void* ptr;
        size_t bytes;
        bool in_graph;
    };
    Block* find(int dev, Stream stream) {
        for (Block& b : blocks_)
            if (b.dev == dev && b.stream == stream) return &b;
        return nullptr;
    }
    std::vector<Block> blocks_;
};

// One mutex for each (device, stream). A call holds it from the lookup of its scratch
// until its last launch is enqueued: its launches hand over through that scratch,
// so those of another thread's call on the stream must not come between them, nor
// may that call's lookup release the block before they are enqueued.
template <class Stream>
class StreamLocks {
   public:
    std::unique_lock<std::mutex> hold(int dev, Stream stream) { return std::unique_lock<std::mutex>(of(dev, stream)); }

   private:
    struct Entry {
        Entry(int d, Stream s) : dev(d), stream(s) {}
        int dev;
        Stream stream;
        std::mutex mu;
    };
    std::mutex& of(int dev, Stream stream) {
        std::lock_guard<std::mutex> lk(mu_);
        for (Entry& e : entries_)
            if (e.dev == dev && e.stream == stream) return e.mu;
        entries_.emplace_back(dev, stream);
        return entries_.back().mu;  // (a deque's elements stay where they are)
    }
    std::mutex mu_;
    std::deque<Entry> entries_;
};

}  // namespace mxw
