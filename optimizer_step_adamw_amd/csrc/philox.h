// philox.h -- the counter-based generator that dropout masks are drawn from:
// Philox4x32-10 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2,
// 3", SC 2011), and a mask's numbers in it.  Plain arithmetic, here so that it
// is checked on the CPU as well.
#pragma once

#include <cstdint>

namespace optim {

struct Words {
    uint32_t w[4];
};

constexpr Words philox(uint64_t block, uint32_t step, uint32_t site, uint64_t seed) {
    uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = step, d = site;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int r = 0; r < 10; ++r) {
        const uint64_t x = (uint64_t)a * 0xD2511F53u, y = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(y >> 32) ^ b ^ k0;
        b = (uint32_t)y;
        c = (uint32_t)(x >> 32) ^ d ^ k1;
        d = (uint32_t)x;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Words{{a, b, c, d}};
}

// Dropout as a kernel takes it.
struct DropArgs {
    uint64_t seed;
    int64_t first;         // place of element 0
    const int32_t *step;   // device, or NULL for 0
    uint32_t site;
    uint32_t bar;          // elements whose 16 bits are below it are dropped; 0: none
    float scale;           // of the others
};

// The 16 bits of the elements at places q .. q + 7: element i's are the low
// (even i) or high half of word i / 2.  Eight places that begin at a multiple of
// eight are one block of the generator, others lie in two.
constexpr Words draws8(uint64_t q, uint32_t step, uint32_t site, uint64_t seed) {
    Words lo = philox(q >> 3, step, site, seed);
    const uint32_t s = (uint32_t)q & 7u;
    if (s == 0) return lo;
    const Words hi = philox((q >> 3) + 1, step, site, seed);
    uint32_t w[8] = {lo.w[0], lo.w[1], lo.w[2], lo.w[3], hi.w[0], hi.w[1], hi.w[2], hi.w[3]};
    if (s & 4u)
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (s & 2u)
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (s & 1u)
        for (int i = 0; i < 4; ++i) w[i] = w[i] >> 16 | w[i + 1] << 16;
    return Words{{w[0], w[1], w[2], w[3]}};
}

constexpr uint32_t draw_of(const Words &w, int i) { return i & 1 ? w.w[i / 2] >> 16 : w.w[i / 2] & 0xFFFFu; }

}  // namespace optim
