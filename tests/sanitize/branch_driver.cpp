// Host-only exercise of the branching operators' entry points, built with AddressSanitizer
// and UndefinedBehaviorSanitizer by tests/test_branch_sanitizers.py: workspace sizes of every
// layout, and device calls only with arguments that they refuse before any launch.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "../../include/cgtp.h"

static int g_fail = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                        \
    }                                                                  \
  } while (0)

int main() {
  alignas(256) static float buf[1024];
  const int32_t* off = reinterpret_cast<const int32_t*>(buf);
  size_t bytes = 1;
  for (int64_t width : {int64_t(1), int64_t(37), int64_t(4096), int64_t(4099), int64_t(1) << 24})
    for (int64_t groups : {int64_t(1), width})
      for (int64_t rows : {int64_t(0), int64_t(1), int64_t(418), int64_t(200000), (int64_t(1) << 31) - 1})
        for (int64_t samples : {int64_t(0), int64_t(1), int64_t(600)})
          for (int64_t longest : {int64_t(0), int64_t(1), rows, int64_t(1) << 40})
            for (int dtype : {CGTP_F32, CGTP_BF16, CGTP_F16})
              for (int backward : {0, 1}) {
                EXPECT(cgtp_group_norm_workspace_size(backward, dtype, rows, width, groups, samples, off, longest,
                                                      &bytes) == CGTP_OK &&
                       bytes % 256 == 0);
                const bool equal = samples ? rows % samples == 0 : rows == 0;
                EXPECT(cgtp_group_norm_workspace_size(backward, dtype, rows, width, groups, samples, nullptr, longest,
                                                      &bytes) == (equal ? CGTP_OK : CGTP_ERR_INVALID_ARG));
              }
  EXPECT(cgtp_group_norm_workspace_size(0, 0, int64_t(1) << 62, 8, 1, 1, nullptr, 0, &bytes) == CGTP_ERR_UNSUPPORTED);
  EXPECT(cgtp_group_norm_workspace_size(0, 0, 1, int64_t(1) << 62, 1, 1, nullptr, 0, &bytes) == CGTP_ERR_UNSUPPORTED);
  EXPECT(cgtp_group_norm_workspace_size(0, 0, 1, 8, int64_t(1) << 62, 1, nullptr, 0, &bytes) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_group_norm_workspace_size(0, 0, 1, 8, 1, int64_t(1) << 62, off, 0, &bytes) == CGTP_ERR_UNSUPPORTED);
  EXPECT(cgtp_group_norm_workspace_size(0, 7, 1, 8, 1, 1, nullptr, 0, &bytes) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_group_norm_workspace_size(0, 0, 1, 8, 1, 1, nullptr, 0, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_group_norm_forward(CGTP_F32, 100000, 8, 2, 1, nullptr, 0, buf, 8, CGTP_F32, nullptr, nullptr, CGTP_ACT_SILU,
                                 1e-5, 0, buf, 8, nullptr, nullptr, 0, nullptr) == CGTP_ERR_WORKSPACE);
  EXPECT(std::strstr(cgtp_last_error(), "workspace") != nullptr);
  EXPECT(cgtp_group_norm_forward(CGTP_F32, 2, 8, 2, 1, nullptr, 0, buf, 8, CGTP_F32, nullptr, nullptr, 9, 1e-5, 0, buf, 8,
                                 nullptr, nullptr, 0, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_group_norm_forward(CGTP_F32, 2, 8, 2, 1, nullptr, 0, buf, 8, CGTP_F32, nullptr, nullptr, 0, std::nan(""), 0,
                                 buf, 8, nullptr, nullptr, 0, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_group_norm_backward(CGTP_F32, 100000, 8, 2, 1, nullptr, 0, buf, 8, buf, 8, buf, CGTP_F32, nullptr, nullptr, 0,
                                  buf, 8, nullptr, nullptr, buf, 16, nullptr) == CGTP_ERR_WORKSPACE);
  EXPECT(cgtp_group_norm_backward(CGTP_F32, 2, 8, 2, 1, nullptr, 0, buf, 8, buf, 8, buf, CGTP_F32, nullptr, nullptr, 0,
                                  nullptr, 8, nullptr, nullptr, nullptr, 0, nullptr) == CGTP_OK);
  for (int n : {1, 8, 17, 1024})
    for (int64_t rows : {int64_t(0), int64_t(1), int64_t(10000), (int64_t(1) << 31) - 1})
      EXPECT(cgtp_route_workspace_size(rows, n, &bytes) == CGTP_OK && bytes % 256 == 0 && (bytes > 0) == (rows > 4096));
  EXPECT(cgtp_route_workspace_size(1, 0, &bytes) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_route_workspace_size(1, 2000, &bytes) == CGTP_ERR_UNSUPPORTED);
  int32_t ids[8];
  EXPECT(cgtp_route_forward(CGTP_F32, 2, 4, 5, buf, 4, nullptr, 0, 0, ids, buf, ids, buf, buf, buf, 4096, nullptr) ==
         CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_route_forward(CGTP_F32, 100000, 4, 2, buf, 4, nullptr, 0, 0, ids, buf, ids, buf, buf, nullptr, 0, nullptr) ==
         CGTP_ERR_WORKSPACE);
  EXPECT(cgtp_route_backward(CGTP_F32, 2, 4, 2, buf, 4, 0, 0, ids, nullptr, nullptr, buf, buf, 4, nullptr) ==
         CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_route_backward(CGTP_F32, 0, 4, 2, nullptr, 4, 0, 0, nullptr, nullptr, nullptr, nullptr, nullptr, 4, nullptr) ==
         CGTP_OK);
  EXPECT(cgtp_conv_gate_backward(2, 4, buf, nullptr, nullptr, buf, buf, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_conv_gate_backward(0, 4, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == CGTP_OK);
  if (g_fail == 0) std::printf("all checks passed\n");
  return g_fail != 0;
}
