// The sequences' own tokens of arc_kv_attend_shared: attention over what lies behind the prefix.
#include "kv_attend.cuh"
#include "kv_shared.cuh"

namespace arcs {

int launch_behind(const arc_kv_cache& cache, const arc_kv_step& step, const arc_kv_query& query, uint32_t* err_word,
                  void* workspace, const SharedLayout& at, int64_t prefix_tokens, int dev, int sms, cudaStream_t st) {
    AttendArgs a = attend_args(cache, step, query, err_word, workspace);
    a.front = static_cast<int32_t>(prefix_tokens);
    a.rows = reinterpret_cast<float*>(static_cast<char*>(workspace) + at.rows);
    a.logs = reinterpret_cast<float*>(static_cast<char*>(workspace) + at.logs);
    return launch_attend<kBehind>(a, dev, sms, st);
}

}  // namespace arcs
