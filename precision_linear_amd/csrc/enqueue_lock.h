// Keeps the launches of one call together (host code).
#pragma once

#include <stdint.h>

#include <mutex>

namespace fp8mm {

// Held while a call enqueues launches that hand each other results through
// `workspace`: host threads that share a stream share its workspace, and another
// call's launch between two of these would write over what the second reads.
// (Calls of one launch need none: the stream orders them.)  The workspace's
// address picks one of 64 locks, so that threads of different streams seldom meet.
inline std::mutex& enqueue_lock(const void* workspace) {
    static std::mutex locks[64];
    return locks[((uint64_t)(uintptr_t)workspace * 0x9E3779B97F4A7C15ull) >> 58];
}

}  // namespace fp8mm
