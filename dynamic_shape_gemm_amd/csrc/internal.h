// What the C-ABI's source files share: error reporting and the launch trace.
#pragma once

#include <hip/hip_runtime.h>
#include <exception>
#include <functional>
#include <string>

#include "../../include/mkp.h"

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

// Trace codes kTraceQ8 - i: the i-th launch of the 8-bit matrices.
constexpr int kTraceQ8 = -40;
enum Q8Launch : int { QL_QUANTIZE, QL_DEQUANTIZE, QL_PACK, QL_I8_PRODUCT, QL_I8_FINISH, QL_SLOPES, QL_Q8_PRODUCT, QL_Q8_FINISH, QL_COUNT };
const char* q8_launch_name(int i);

// No exception leaves the C entry points.
template <class F>
int guarded(F&& fn) {
    try {
        return fn();
    } catch (const std::exception& e) {
        try {
            return report(MKP_ERR_HIP, e.what());
        } catch (...) {
        }
    } catch (...) {
    }
    return MKP_ERR_HIP;
}

}  // namespace mkp
