// Heads of every kind, among them whatever stood in memory: those that join_in_reach accepts lead the join nowhere but
// into its buffers, and those that a division into chunks gives are accepted.
#include <cstdio>
#include <cstring>
#include <random>

#include "../fp8_block_scaled_fp8bs_gb300/csrc/attention_join.h"

int main() {
    std::mt19937_64 rng(1);
    auto below = [&](int64_t n) { return static_cast<int64_t>(rng() % static_cast<uint64_t>(n)); };
    long violations = 0, accepted = 0;
    const int forms[] = {8, 16, 32};
    for (int n = 0; n < 4000000; ++n) {
        const int most = forms[below(3)];
        const int64_t group = 1 + below(n & 2 ? most : 65535), tokens = 1 + below(n & 1 ? 300 : 2147483647);
        const int64_t chunks = 1 + below(n & 4 ? 1300 : 2147483647);
        fp8bs::JoinHead j;
        int* field[] = {&j.parts, &j.first, &j.q0, &j.rows};
        for (int i = 0; i < 4; ++i) {
            const int64_t kind = below(6);
            const int64_t range[] = {chunks, chunks, tokens, most};
            const uint32_t any = static_cast<uint32_t>(rng());
            int32_t word;
            std::memcpy(&word, &any, 4);
            *field[i] = kind == 0 ? word : kind == 1 ? static_cast<int>(below(5)) - 2
                                                     : static_cast<int>(below(range[i] + 2)) - (kind == 2 ? 1 : 0);
        }
        if (!fp8bs::join_in_reach(j, chunks, most, group, tokens)) continue;
        ++accepted;
        // parts: 2 slots of `most` rows in each chunk; marks of them; rows of the output
        const __int128 last = static_cast<__int128>(j.first) + j.parts - 1;
        const __int128 row = static_cast<__int128>(j.q0) * group + j.rows - 1;
        if (j.parts < 1 || j.first < 0 || last >= chunks || j.rows < 1 || j.rows > most || j.q0 < 0 ||
            row >= static_cast<__int128>(tokens) * group)
            ++violations;
    }
    long refused = 0;
    for (int n = 0; n < 1000000; ++n) {
        const int most = forms[below(3)];
        const int64_t group = 1 + below(most), tokens = 1 + below(100000), chunks = 2 + below(1300);
        const int64_t news = 1 + below(most / group < tokens ? most / group : tokens);
        fp8bs::JoinHead j;
        j.first = static_cast<int>(below(chunks - 1));
        j.parts = 2 + static_cast<int>(below(chunks - 1 - j.first));
        j.rows = static_cast<int>(news * group);
        j.q0 = static_cast<int>(below(tokens - news + 1));
        refused += !fp8bs::join_in_reach(j, chunks, most, group, tokens);
    }
    std::printf("accepted %ld violations %ld refused %ld\n", accepted, violations, refused);
    return violations || refused || accepted < 1000;
}
