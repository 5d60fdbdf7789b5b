// Device status codes written to the context's status word, and wait limits.
#pragma once
#include <cstdint>

namespace lora {

// A bounded device wait gives up after this long (nanoseconds of %globaltimer).
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// What a kernel found; the status word has bit 1 << code of every code raised since it was
// last read.
enum DeviceStatus : unsigned {
    kDevOk = 0,
    kDevTimeoutLoad = 1,   // a copy into shared memory did not complete in time
    kDevTimeoutMma = 2,    // a tensor-core commit did not arrive in time
    kDevTimeoutPipe = 3,   // a producer/consumer pipeline slot was not released
    kDevBadShape = 4,      // a kernel found a size it cannot handle (skipped)
    kDevBadId = 5,         // a device-resident adapter id the table cannot serve (row skipped)
    kDevBadBatch = 6,      // a sequence's rows or length out of range (sequence skipped)
    kDevBadPage = 7        // a page id outside the cache's pools (its positions skipped)
};

// The codes after which a kernel has left work undone (bits of the status word).
constexpr unsigned kDevGaveUp = 1u << kDevTimeoutLoad | 1u << kDevTimeoutMma | 1u << kDevTimeoutPipe | 1u << kDevBadShape;

}  // namespace lora
