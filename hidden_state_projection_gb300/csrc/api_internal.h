// api_internal.h -- what the C entry points of other files share with proj_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "proj.h"

namespace hsp {

// Sets the text of proj_last_error_string and returns `st`.
proj_status api_fail(proj_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
proj_status api_cuda_fail(cudaError_t e, const char *what);
proj_status api_ok();

// The current device: refused unless compute capability 10.3.
struct ApiDevice {
    int sms;
    int *err_word;
};
proj_status api_device(ApiDevice *out);
// SM count of the current device, 152 where there is none (host-only queries).
int api_plan_sms();

// Options a launch takes its behaviour from.
struct ApiOptions {
    int pdl;
    int skip_stage;  // -1: off
    uint64_t wait_limit_ns;
};
ApiOptions api_options();
void api_count_launches(int n);

// Tiled bf16 tensor map of five dimensions (128-byte swizzle, zero fill), made anew per call.
proj_status api_encode_5d(const void *ptr, const uint64_t (&dims)[5], const uint64_t (&strides)[4],
                          const uint32_t (&box)[5], CUtensorMap *out);
// The same of bytes, boxes 128 or 64 columns wide (128- or 64-byte swizzle).
proj_status api_encode_codes_5d(const void *ptr, const uint64_t (&dims)[5], const uint64_t (&strides)[4],
                                const uint32_t (&box)[5], bool joined, CUtensorMap *out);

}  // namespace hsp
