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
// what the join reads and writes is within its buffers then, whatever else the head says.
FP8BS_BOTH inline bool join_in_reach(const JoinHead& j, int64_t chunks, int64_t most, int64_t group, int64_t tokens) {
    return j.parts > 0 && j.first >= 0 && static_cast<int64_t>(j.first) + j.parts <= chunks && j.rows > 0 &&
           j.rows <= most && j.q0 >= 0 && j.q0 + (j.rows - 1) / group < tokens;
}

}  // namespace fp8bs
