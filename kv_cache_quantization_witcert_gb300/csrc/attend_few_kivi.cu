#include "attend_few.cuh"

namespace witcert {

template cudaError_t launch_attend_few<kKivi>(const AttendArgs&, cudaStream_t);

}  // namespace witcert
