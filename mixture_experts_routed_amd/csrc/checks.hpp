// Argument checks shared by the C ABI's translation units (host only).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_routed.h"

namespace {

constexpr int64_t kI32Max = 2147483647;

bool aligned(const void *p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_F16 || dtype == MOE_BF16; }

hipStream_t as_stream(moe_stream_t s) { return static_cast<hipStream_t>(s); }

}  // namespace
