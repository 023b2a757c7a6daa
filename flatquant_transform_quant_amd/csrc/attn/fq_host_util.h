// Checks and error reporting shared by the host files of the library (fq_host.cpp defines them).
#pragma once

#include <hip/hip_runtime.h>

#include "fq.h"

namespace fq {

bool is_contiguous(const fq_tensor& t);
// at most 4 dimensions, no negative size or stride
bool strides_ok(const fq_tensor& t);
bool shape_is(const fq_tensor& t, int nd, int64_t a, int64_t b = 0, int64_t c = 0);

// fq_last_error()'s text, per host thread
void clear_last_error();
const char* last_error();
void set_last_error(const char* fmt, unsigned long long a, unsigned long long b);
fq_status fail_runtime(const char* what, hipError_t err);

bool device_is_gfx950();

}  // namespace fq
