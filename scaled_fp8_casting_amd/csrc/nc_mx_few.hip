// The few-row product by its operands' formats.
#include "nc_mx_few.h"

namespace nc {

hipError_t launch_mx_few(const MxProduct& p, int fa, int fb, int t, hipStream_t stream) {
  return fa == NC_E2M1 ? mx_few_e2m1(p, fb, t, stream) : fa == NC_E4M3 ? mx_few_e4m3(p, fb, t, stream) : mx_few_e5m2(p, fb, t, stream);
}

}  // namespace nc
