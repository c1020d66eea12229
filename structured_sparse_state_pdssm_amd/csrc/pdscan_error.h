// The calling thread's error text (pdssm_last_error), set by every entry point.
#pragma once

namespace pdscan {

int set_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));   // returns code
void clear_error();

}  // namespace pdscan
