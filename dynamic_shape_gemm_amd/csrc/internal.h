// What the C-ABI's source files share: error reporting and the launch trace.
#pragma once

#include <hip/hip_runtime.h>
#include <functional>
#include <string>

namespace mkp {

// Sets this thread's error message and returns `code`.
int report(int code, const std::string& msg);

// Starts a C-ABI call: the sequence number its launches carry in the trace.
void begin_call();

// Runs one launch, timed in trace mode under kernel code `kernel`.
hipError_t traced_launch(hipStream_t st, int kernel, double flops, double bytes,
                         const std::function<hipError_t()>& fn);

// Trace codes kTraceLoss - i: the i-th launch of the vocabulary losses.
constexpr int kTraceLoss = -20;
enum LossLaunch : int { LL_FLAGS, LL_SCAN, LL_GATHER, LL_FORWARD, LL_FINISH, LL_GRAD, LL_PRODUCTS, LL_OUTPUTS, LL_COUNT };
const char* loss_launch_name(int i);

}  // namespace mkp
