// attend_sinks.cu -- attention of new tokens that see a window and first tokens that stay visible.
#include "attend_set.cuh"

namespace up {

cudaError_t launch_attend_sinks(const AttendArgs &a, int num_sms, cudaStream_t st) {
    return launch_set<kSinks>(a, num_sms, st);
}

}  // namespace up
