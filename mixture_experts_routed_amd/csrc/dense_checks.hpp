// Argument checks shared by the C ABI of the dense operators and of those around the
// block (host only).
#pragma once

#include <initializer_list>

#include "checks.hpp"

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 20;  // row lengths and strides, elements

// a row-major [*][cols] operand with row stride ld
bool rows_ok(int64_t cols, int64_t ld) { return ld >= cols && ld <= kMaxCols; }

// an array that may be left out
bool aligned_or_null(const void *p, size_t a) { return !p || aligned(p, a); }

bool result_ok(int dtype, int operand) { return dtype == MOE_F32 || dtype == operand; }

// an output that may be one of the inputs: element by element, so with the same stride
bool in_place_ok(const void *out, int64_t ldo, const void *in, int64_t ldi, int T)
{
    return !in || out != in || ldo == ldi || T == 1;
}

// outputs that are asked for lie apart
bool apart(const void *a, const void *b) { return !a || a != b; }

// an output that is asked for is none of a call's other arguments
bool apart_from(const void *out, std::initializer_list<const void *> others)
{
    for (const void *p : others)
        if (!apart(out, p)) return false;
    return true;
}

bool workspace_ok(const void *p, size_t have, size_t need)
{
    return need == 0 || (aligned(p, 256) && have >= need);
}

}  // namespace
