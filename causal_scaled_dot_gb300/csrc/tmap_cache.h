// tmap_cache.h -- caches of encoded TMA tensor maps: a small one that is searched from end to end, and
// a larger one whose keys are hashed to sets.  Both replace the least recently used entry, of all or of the set.
//
// A tiled tensor map is a pure function of what the encoder is given: the base
// address, the element type, the extents, the strides and the box.  The key
// below holds every one of those inputs (strides follow from the extents for
// the contiguous views this library encodes) plus the device, so a hit always
// returns exactly the map a fresh encode would produce.  That makes the cache
// safe against reused addresses: a buffer that is freed and reallocated at the
// same address with the same geometry gets the same map, which is correct for
// it; any change of address, geometry or box is a different key.
//
// Not thread-safe by itself: the caller serialises lookup/insert (attn_api.cu
// holds a mutex around them).  Header-only and free of CUDA runtime calls, so
// host tests can compile it with a plain C++ compiler.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <cstring>

namespace attn {

struct TmapKey {
    int device;
    const void* ptr;
    int elem_bytes;
    int D;
    int S;
    long long outer;
    int box_rows;

    bool operator==(const TmapKey& o) const {
        return device == o.device && ptr == o.ptr && elem_bytes == o.elem_bytes && D == o.D && S == o.S &&
               outer == o.outer && box_rows == o.box_rows;
    }
};

template <int N>
class TmapCache {
  public:
    // On a hit copies the cached map into *map and returns true.
    bool lookup(const TmapKey& key, CUtensorMap* map) {
        for (int i = 0; i < N; ++i) {
            if (used_[i] != 0 && keys_[i] == key) {
                std::memcpy(map, &maps_[i], sizeof(CUtensorMap));
                used_[i] = ++clock_;
                ++hits_;
                return true;
            }
        }
        ++misses_;
        return false;
    }
    // Stores a freshly encoded map, replacing the least recently used entry.
    void insert(const TmapKey& key, const CUtensorMap& map) {
        int victim = 0;
        for (int i = 0; i < N; ++i) {
            if (used_[i] == 0) {
                victim = i;
                break;
            }
            if (used_[i] < used_[victim]) victim = i;
        }
        keys_[victim] = key;
        std::memcpy(&maps_[victim], &map, sizeof(CUtensorMap));
        used_[victim] = ++clock_;
    }
    unsigned long long hits() const { return hits_; }
    unsigned long long misses() const { return misses_; }

  private:
    TmapKey keys_[N] = {};
    CUtensorMap maps_[N] = {};
    unsigned long long used_[N] = {};  // 0: empty slot; otherwise the last use's clock
    unsigned long long clock_ = 0;
    unsigned long long hits_ = 0, misses_ = 0;
};

// `Sets` sets (a power of two) of `Ways` entries each: for callers with many buffers, such as a model's
// layers, each with tensors of its own, where a search of everything would cost more than a map's encoding.
template <int Sets, int Ways>
class TmapTable {
    static_assert(Sets > 0 && (Sets & (Sets - 1)) == 0, "a power of two");

  public:
    bool lookup(const TmapKey& key, CUtensorMap* map) { return sets_[set_of(key)].lookup(key, map); }
    void insert(const TmapKey& key, const CUtensorMap& map) { sets_[set_of(key)].insert(key, map); }

  private:
    // Every field counts, the address by its multiples of 16 (a multiplication's upper bits depend on all bits below).
    static int set_of(const TmapKey& k) {
        unsigned long long h = (unsigned long long)(uintptr_t)k.ptr >> 4;
        const unsigned long long rest[4] = {(unsigned long long)(unsigned)k.device * 8 + (unsigned)k.elem_bytes,
                                            (unsigned long long)(unsigned)k.D * 512 + (unsigned)k.box_rows, (unsigned long long)(unsigned)k.S,
                                            (unsigned long long)k.outer};
        for (unsigned long long x : rest) h = (h ^ x) * 0x9E3779B97F4A7C15ull;
        h ^= h >> 32;
        h *= 0x9E3779B97F4A7C15ull;
        return (int)(h >> 40) & (Sets - 1);
    }
    TmapCache<Ways> sets_[Sets];
};

}  // namespace attn
