// norm_rotary.h -- how norm_rotary_kernel's work is cut into CTAs (host).
#pragma once

#include <algorithm>

#include "rotary_common.cuh"

namespace kvevict {

constexpr int kNormStages = 4;
constexpr int kNormPairs = 256;  // of a head of 64 chunks at most

// Four CTAs an SM: their registers are the launch bound's, and of its 228 KB of shared
// memory (1 KB of a CTA is not its own) the stages of loads, the frequencies, and the
// table of cosines, which is what is left.
constexpr int kNormCtas = 4, kNormSlots = kNormCtas * 152;
constexpr int kNormOwn = kNormStages * 2 * kRotThreads * 16;
constexpr int kNormTable = (228 * 1024) / kNormCtas - 1024 - kNormPairs * 8 - kNormOwn;

// A CTA's share of tokens (all heads): what lets whole waves of four CTAs an SM end
// soonest, a CTA taking what its rows take and as much as kNormStart times its 256
// threads' rows to find its way and its cosines. (16384 tokens, 64 + 8 heads of 128:
// 108 us, 82% of the copy bandwidth, 111 with 4 tokens a CTA; 3 x 2049 tokens, 12 + 4
// heads, 48 of 128 in fp32: 26 us, 30 with ten tokens a CTA; 32768 tokens of
// 64 + 8 heads: 199 us, 238 with 54 tokens a CTA, of which three fit an SM.)
constexpr int kNormStart = 5;

inline int norm_tokens(long long total, long long heads, long long step, int R)
{
    int best = 1;
    double least = 0;
    for (int t = 1; t <= std::min(64, kNormTable / (std::max(R, 2) / 2 * 8)); ++t) {
        const long long waves = ((total + t - 1) / t + kNormSlots - 1) / kNormSlots;
        const double cost = static_cast<double>(waves) * (static_cast<double>(t * heads) / static_cast<double>(step) + kNormStart);
        if (t == 1 || cost < least * 0.995) {
            least = cost;
            best = t;
        }
    }
    return best;
}

}  // namespace kvevict
