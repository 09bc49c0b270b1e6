// The library's status reporting, shared by the files that hold C entry points.
#pragma once

namespace q4 {

// Keep `msg` as this thread's q4_last_error() text and return `code`.
int report(int code, const char* msg) noexcept;

}  // namespace q4
