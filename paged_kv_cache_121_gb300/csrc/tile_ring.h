// Slots of shared memory that tiles are fetched into, one after another, and which of them
// still have a copy on its way. Plain C++: the counting can be run on the host.
#pragma once

#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif

namespace pa {

struct TileRing {
    int slots;
    int sent = 0;   // tiles whose copies were issued

    PA_HOST_DEVICE explicit TileRing(int n) : slots(n) {}
    PA_HOST_DEVICE int slot() const { return sent % slots; }   // of the next tile
    // Parity of the `empty` phase that the next tile waits for; negative: its slot has not been used yet.
    PA_HOST_DEVICE int empty_parity() const {
        const int round = sent / slots;
        return round > 0 ? (round - 1) & 1 : -1;
    }
    // A tile whose wait ran out was not sent: nothing of it will arrive.
    PA_HOST_DEVICE void count(bool issued) { sent += issued ? 1 : 0; }
    // Tiles first_left .. sent - 1 may be on their way (an older one has left its slot, so it has arrived); tile n
    // arrives in slot n % slots, in the phase of this parity.
    PA_HOST_DEVICE int first_left() const { return sent > slots ? sent - slots : 0; }
    PA_HOST_DEVICE int full_parity(int n) const { return (n / slots) & 1; }
};

}  // namespace pa
