// arc_kv_attend: causal attention of a step's new tokens, optionally within a window.
#include "kv_attend.cuh"

extern "C" {

size_t arc_kv_attend_workspace_bytes(const arc_kv_cache* cache) {
    return check_cache(cache) == ARC_OK ? attend_workspace(*cache) : 0;
}

int arc_kv_attend(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query, uint32_t* err_word,
                  void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_attend(cache, step, query, err_word);
    if (rc != ARC_OK) return rc;
    if (workspace == nullptr || workspace_bytes < attend_workspace(*cache)) return ARC_E_WORKSPACE;
    if (!aligned(workspace, 16)) return ARC_E_ALIGN;
    int dev = 0, sms = 0;
    rc = device_of(dev, sms);
    if (rc != ARC_OK) return rc;
    return launch_attend<kPlain>(attend_args(*cache, *step, *query, err_word, workspace), dev, sms,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"
