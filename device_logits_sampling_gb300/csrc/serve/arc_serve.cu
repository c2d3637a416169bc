// Names of libarcserve's return codes, and its version.
#include "serve/arc_kv.h"

extern "C" {

const char* arc_serve_strerror(int code) {
    switch (code) {
        case ARC_OK: return "ok";
        case ARC_E_NULL: return "a required pointer is NULL";
        case ARC_E_SHAPE: return "a size, stride or count is out of range";
        case ARC_E_DTYPE: return "unsupported element type";
        case ARC_E_ALIGN: return "a pointer or stride is not aligned as the call needs";
        case ARC_E_UNSUPPORTED: return "unsupported head size, page size or group";
        case ARC_E_OPTION: return "an option (layout, amplitude, scale, window, reserved field) is invalid";
        case ARC_E_CUDA: return "CUDA error while configuring or launching";
        case ARC_E_WORKSPACE: return "workspace is NULL or too small";
        default: return "unknown error code";
    }
}

int arc_serve_abi_version(void) { return ARC_SERVE_ABI_VERSION; }

}  // extern "C"
