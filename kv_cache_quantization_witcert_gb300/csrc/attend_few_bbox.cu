#include "attend_few.cuh"

namespace witcert {

template cudaError_t launch_attend_few<kBbox>(const AttendArgs&, cudaStream_t);

}  // namespace witcert
