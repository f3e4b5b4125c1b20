// Host-side helpers that the C entry points share (defined in cgtp_api.hip): the
// thread-local error message and the irreps parser.
#pragma once

#include <hip/hip_runtime.h>

#include <string>
#include <vector>

namespace cgtp {

// Sets the thread's message and returns `code`.
int fail(int code, const char* fmt, ...);
// Clears the thread's message and returns CGTP_OK.
int ok();

#define CGTP_HIP(call)                                                                  \
  do {                                                                                  \
    hipError_t e_ = (call);                                                             \
    if (e_ != hipSuccess) return fail(CGTP_ERR_HIP, "%s: %s", #call, hipGetErrorString(e_)); \
  } while (0)

struct Irrep {
  int mul, l, p;
};

// Parse "128x0e+64x1o" (a bare "1o" means multiplicity 1).
bool parse_irreps(const char* spec, std::vector<Irrep>& out, std::string& err);

}  // namespace cgtp
