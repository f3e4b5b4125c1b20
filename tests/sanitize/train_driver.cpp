// Host-only exercise of the training operators' entry points, built with AddressSanitizer
// and UndefinedBehaviorSanitizer by tests/test_train_sanitizers.py: plans and sets without
// a device, and device calls only with arguments that they refuse before any launch.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

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
  size_t bytes = 1;
  // plans: counts, refusals, and sizes of every layout of short, long and wide stretches
  for (const char* spec : {"1x0e", "16x0e+8x1e+16x1o", "20000x0e+3x1o+7000x1o", "512x6e", "1o"}) {
    cgtp_norm_t p = nullptr;
    EXPECT(cgtp_norm_create(spec, &p) == CGTP_OK && p);
    int64_t f = 0, w = 0, b = 0;
    int t = 0;
    EXPECT(cgtp_norm_info(p, &f, &w, &b, &t) == CGTP_OK && f >= w && w >= b && t > 0);
    EXPECT(cgtp_norm_info(p, nullptr, nullptr, nullptr, nullptr) == CGTP_OK);
    for (int64_t rows : {int64_t(0), int64_t(1), int64_t(7), int64_t(1000), int64_t(1) << 31})
      EXPECT(cgtp_irreps_norm_backward_workspace_size(p, rows, &bytes) == CGTP_OK && bytes % 256 == 0);
    EXPECT(cgtp_irreps_norm_backward_workspace_size(p, -1, &bytes) == CGTP_ERR_INVALID_ARG);
    EXPECT(cgtp_irreps_norm_forward(p, 9, 1, buf, f, 0, nullptr, nullptr, 1e-5, buf, f, nullptr, nullptr) ==
           CGTP_ERR_INVALID_ARG);
    EXPECT(cgtp_irreps_norm_forward(p, CGTP_F32, 0, nullptr, f, 0, nullptr, nullptr, 1e-5, nullptr, f, nullptr,
                                    nullptr) == CGTP_OK);
    cgtp_norm_destroy(p);
  }
  cgtp_norm_t none = nullptr;
  std::string many = "1x0e";
  for (int k = 0; k < 64; ++k) many += "+1x1o";
  EXPECT(cgtp_norm_create(many.c_str(), &none) == CGTP_ERR_UNSUPPORTED && !none);
  EXPECT(cgtp_norm_create("4x0", &none) == CGTP_ERR_PARSE && cgtp_norm_create(nullptr, &none) == CGTP_ERR_PARSE);
  EXPECT(cgtp_norm_create("4x9e", &none) == CGTP_ERR_UNSUPPORTED && cgtp_norm_create("4x0e", nullptr) != CGTP_OK);
  cgtp_norm_destroy(nullptr);
  for (int64_t width : {int64_t(1), int64_t(5), int64_t(1024), int64_t(16385), int64_t(1) << 29})
    EXPECT(cgtp_layer_norm_backward_workspace_size(100, width, &bytes) == CGTP_OK);
  EXPECT(cgtp_layer_norm_backward_workspace_size(100, 0, &bytes) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_layer_norm_forward(CGTP_F32, 2, 8, buf, 4, CGTP_F32, nullptr, nullptr, 1e-5, buf, 8, nullptr, nullptr) ==
         CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_layer_norm_backward(CGTP_F32, 1000, 8, buf, 8, buf, 8, buf, CGTP_F32, nullptr, nullptr, 8, buf, nullptr,
                                  nullptr, 0, nullptr) == CGTP_ERR_WORKSPACE);
  // sets: offsets, refusals, device calls without a device
  std::vector<int64_t> sizes;
  std::vector<double> decay;
  int64_t at = 0;
  for (int k = 0; k < 700; ++k) {
    sizes.push_back(k * 37 % 5000);
    decay.push_back(k % 2 ? 0.0 : 0.01);
  }
  cgtp_params_t set = nullptr;
  EXPECT(cgtp_params_create(sizes.data(), decay.data(), int(sizes.size()), CGTP_PLAN_HOST_ONLY, &set) == CGTP_OK);
  std::vector<int64_t> offs(sizes.size());
  int n = 0;
  int64_t elems = 0;
  EXPECT(cgtp_params_info(set, &n, &elems, offs.data()) == CGTP_OK && n == 700);
  for (int k = 0; k < n; ++k) {
    EXPECT(offs[size_t(k)] == at);
    at += (sizes[size_t(k)] + 63) / 64 * 64;
  }
  EXPECT(elems == at);
  EXPECT(cgtp_grad_norm_workspace_size(set, &bytes) == CGTP_OK && bytes > 0);
  std::vector<void*> ptr(sizes.size(), buf);
  EXPECT(cgtp_adamw_step(set, 0, ptr.data(), 0, ptr.data(), buf, buf, 1e-3, 0.9, 0.999, 1e-8, 1, nullptr, nullptr,
                         nullptr) ==
         CGTP_ERR_INVALID_ARG);
  EXPECT(std::strstr(cgtp_last_error(), "HOST_ONLY") != nullptr);
  cgtp_params_destroy(set);
  int64_t step = 0;
  EXPECT(cgtp_adamw_scalars(nullptr, nullptr, 1e-3, 0.9, 0.999, 0, nullptr, buf, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_adamw_scalars(&step, nullptr, -1.0, 0.9, 0.999, 0, nullptr, buf, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_adamw_scalars(&step, nullptr, 1e-3, 1.0, 0.999, 0, nullptr, buf, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_adamw_scalars(&step, nullptr, 1e-3, 0.9, 0.999, 0, nullptr, buf + 1, nullptr) == CGTP_ERR_INVALID_ARG);
  EXPECT(step == 0);
  sizes[3] = -1;
  EXPECT(cgtp_params_create(sizes.data(), nullptr, 5, CGTP_PLAN_HOST_ONLY, &set) == CGTP_ERR_INVALID_ARG && !set);
  sizes[3] = int64_t(1) << 41;
  EXPECT(cgtp_params_create(sizes.data(), nullptr, 5, CGTP_PLAN_HOST_ONLY, &set) == CGTP_ERR_UNSUPPORTED);
  sizes[3] = 5;
  decay[3] = std::nan("");
  EXPECT(cgtp_params_create(sizes.data(), decay.data(), 5, CGTP_PLAN_HOST_ONLY, &set) == CGTP_ERR_INVALID_ARG);
  EXPECT(cgtp_params_create(nullptr, nullptr, 0, CGTP_PLAN_HOST_ONLY, &set) == CGTP_OK);
  cgtp_params_destroy(set);
  cgtp_params_destroy(nullptr);
  if (g_fail == 0) std::printf("all checks passed\n");
  return g_fail != 0;
}
