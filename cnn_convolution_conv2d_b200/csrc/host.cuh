// host.cuh -- what the files with C entry points share (defined in abi.cu).
#pragma once

#include "common.cuh"

namespace conv2d_b200 {

int abi_fail(int status, const char *fmt, ...);  // keeps the message for conv2d_last_error and returns status
int abi_ok();
// Counts the launch, or keeps its error.
int abi_launch(cudaError_t e, const char *what);

struct AbiDevice {
    int sms;
    int *status;            // the device status word conv2d_sync_status reads
    long long timeout_ns;   // limit of a device-side wait
    int starve;             // test hook
};
// The current device; fails on one that this library is not built for.
int abi_device(AbiDevice *out);

// A matrix of `rows` rows of `cols` elements (2 or 4 bytes), rows `row_bytes` apart, as a tiled
// tensor map without swizzle; what lies outside reads as zero and is not written.
int abi_tensor_map_2d(CUtensorMap *map, const void *p, int elt, long long cols, long long rows, long long row_bytes,
                      int box_cols, int box_rows);

}  // namespace conv2d_b200
