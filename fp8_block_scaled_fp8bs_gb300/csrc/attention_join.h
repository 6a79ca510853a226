// attention_join.h -- what the join of parts over a cache of codes (attention_fp8.cu) is told, and whether it may be
// followed. Plain C++, for the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FP8BS_BOTH __host__ __device__
#else
#define FP8BS_BOTH
#endif

namespace fp8bs {

// Where the part that a chunk begins with ends its sequence, what is to be joined.
struct JoinHead {
    int parts;             // 0: nothing
    int first;             // chunk of the first part
    int q0, rows;
};

// Whether the parts stand in `chunks` chunks and the rows among `tokens` tokens of `group` rows each, `most` rows at most:
// what the join reads and writes is within its buffers then, whatever else the head says. (In 32 bits, negative numbers
// as large ones: in 64 one token of 32k keys took 24.6 us instead of 23.6.)
FP8BS_BOTH inline bool join_in_reach(const JoinHead& j, uint32_t chunks, uint32_t most, uint32_t group, uint32_t tokens) {
    const uint32_t parts = static_cast<uint32_t>(j.parts), first = static_cast<uint32_t>(j.first);
    const uint32_t q0 = static_cast<uint32_t>(j.q0), rows = static_cast<uint32_t>(j.rows);
    if (parts - 1 >= chunks || first > chunks - parts || rows - 1 >= most || q0 >= tokens) return false;
    return (tokens - q0 < most ? tokens - q0 : most) * group >= rows;        // (`most` tokens have that many rows)
}

}  // namespace fp8bs
