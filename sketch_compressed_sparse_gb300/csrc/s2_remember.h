// Answers kept by their questions, in a table of fixed size without allocation:
// a set of eight places by the key's hash, of which the oldest is given up. (The
// questions are about shapes, thousands at most in a process; an answer that was
// given up is looked up again.) Callers hold a lock.
#pragma once

#include <cstdint>

namespace s2 {

// Key: operator== and hash(). kSets: a power of two.
template <typename Key, typename Value, uint32_t kSets>
class Remembered {
public:
    bool find(const Key& key, Value* value) const {
        const Set& s = sets_[key.hash() % kSets];
        for (uint32_t i = 0; i < s.used; ++i)
            if (s.keys[i] == key) {
                *value = s.values[i];
                return true;
            }
        return false;
    }
    // (a key that is not there yet)
    void put(const Key& key, const Value& value) {
        Set& s = sets_[key.hash() % kSets];
        const uint32_t i = s.used < kPlaces ? s.used++ : s.oldest++ % kPlaces;
        s.keys[i] = key;
        s.values[i] = value;
    }

private:
    static constexpr uint32_t kPlaces = 8;
    struct Set {
        Key keys[kPlaces];
        Value values[kPlaces];
        uint32_t used, oldest;
    };
    Set sets_[kSets];
};

// Spreads the bits of a word over all of it (a product with an odd constant, its high half folded in, twice).
inline uint64_t spread(uint64_t x) {
    for (int i = 0; i < 2; ++i) {
        x *= 0x9E3779B97F4A7C15ull;
        x ^= x >> 32;
    }
    return x;
}

}  // namespace s2
