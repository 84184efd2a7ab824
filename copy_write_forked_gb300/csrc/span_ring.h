// Where the regions of a ring buffer lie, and which of them are still in use:
// the arithmetic of the staging ring (Staging), without CUDA.
#pragma once

#include <cstddef>
#include <deque>

namespace dendrite {

// Tag: what says that a region is free again (an event).
template <typename Tag>
class SpanRing {
public:
    void reset(size_t cap) {
        cap_ = cap;
        head_ = 0;
        used_.clear();
    }
    size_t cap() const { return cap_; }
    // Offset of the next region of `bytes` <= cap(): behind the last one, or at
    // the start where it would pass the end.  Every region in use that it meets,
    // and every older one, is given to done(tag), oldest first, and is then out
    // of use; done waits for it and returns whether that went well.
    template <typename Done>
    bool place(size_t bytes, size_t* off, Done done) {
        size_t at = head_;
        if (at + bytes > cap_) at = 0;
        size_t meets = 0;
        for (size_t k = 0; k < used_.size(); ++k)
            if (used_[k].off < at + bytes && at < used_[k].end) meets = k + 1;
        for (; meets; --meets) {
            const Tag t = used_.front().tag;
            used_.pop_front();
            if (!done(t)) return false;
        }
        head_ = at + bytes;
        *off = at;
        return true;
    }
    void use(size_t off, size_t bytes, Tag tag) { used_.push_back({off, off + bytes, tag}); }
    // Every region in use, oldest first, to done(tag).
    template <typename Done>
    void drain(Done done) {
        for (const Region& r : used_) done(r.tag);
        used_.clear();
    }

private:
    struct Region {
        size_t off, end;
        Tag tag;
    };
    size_t cap_ = 0, head_ = 0;
    std::deque<Region> used_;
};

}  // namespace dendrite
