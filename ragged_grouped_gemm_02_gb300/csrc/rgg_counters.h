// rgg_counters.h -- which set of a handle's tile counters a launch with claims
// (rgg_sched.cuh) takes.
//
// Two launches may use one set only where the second starts after the first
// has ended, which a stream promises for its own launches.  So a set belongs to
// one stream, by the identifier that is never used again for another stream
// (its pointer may be), and within a capture to one stream of that capture, by
// its pointer and the capture's identifier: a graph's launches run wherever the
// graph does, beside what the stream they were captured from does meanwhile.
// A set is never given back: nothing says when a stream's or a graph's last
// launch has ended.  Where all are taken the caller launches without claims.
#pragma once

#include <cstdint>
#include <mutex>

namespace rgg {

constexpr int kCounterSets = 4096;
constexpr int kCounterSetWords = 8;  // three are used; a set fills a 32-byte sector

class CounterSets {
public:
    // The set of this stream and capture (0: none), or -1 where all sets are others'.
    int set_of(uint64_t stream, uint64_t capture) {
        std::lock_guard<std::mutex> lock(mutex_);
        const uint64_t mixed = (stream * 0x9E3779B97F4A7C15ull) ^ (capture * 0xC2B2AE3D27D4EB4Full);
        const int first = static_cast<int>((mixed >> 32) % kCounterSets);
        for (int i = 0; i < kCounterSets; ++i) {
            Owner& o = owner_[(first + i) % kCounterSets];
            if (!o.taken) o = Owner{stream, capture, true};
            if (o.stream == stream && o.capture == capture) return (first + i) % kCounterSets;
        }
        return -1;
    }

private:
    struct Owner {
        uint64_t stream, capture;
        bool taken;
    };
    std::mutex mutex_;
    Owner owner_[kCounterSets] = {};
};

}  // namespace rgg
