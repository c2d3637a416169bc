// arc_kv_attend_sinks: attention within a window, with a sequence's first tokens always visible.
#include "kv_attend.cuh"

extern "C" int arc_kv_attend_sinks(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query,
                                   int32_t sinks, uint32_t* err_word, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    int rc = check_attend(cache, step, query, err_word);
    if (rc != ARC_OK) return rc;
    if (sinks < 0) return ARC_E_OPTION;
    // without a window every token is visible, without sinks the window's alone
    if (sinks == 0 || query->window == 0)
        return arc_kv_attend(cache, step, query, err_word, workspace, workspace_bytes, stream);
    if (workspace == nullptr || workspace_bytes < attend_workspace(*cache)) return ARC_E_WORKSPACE;
    if (!aligned(workspace, 16)) return ARC_E_ALIGN;
    int dev = 0, sms = 0;
    rc = device_of(dev, sms);
    if (rc != ARC_OK) return rc;
    AttendArgs a = attend_args(*cache, *step, *query, err_word, workspace);
    a.front = sinks;
    return launch_attend<kSinks>(a, dev, sms, static_cast<cudaStream_t>(stream));
}
