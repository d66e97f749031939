// What the library's translation units share on the host side.
#pragma once

#include <cstddef>

constexpr size_t kErrorText = 512;

// The calling thread's message for its last nonzero return (zero_last_error).
__attribute__((visibility("hidden"))) char* zero_error_text();
