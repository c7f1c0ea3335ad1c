// Products with few rows whose first operand is E2M1.
#include "nc_mx_few.h"

namespace nc {

hipError_t mx_few_e2m1(const MxProduct& p, int fb, int t, hipStream_t stream) {
  return fb == NC_E2M1 ? mx_few_launch<NC_E2M1, NC_E2M1>(p, t, stream)
       : fb == NC_E4M3 ? mx_few_launch<NC_E2M1, NC_E4M3>(p, t, stream)
                       : mx_few_launch<NC_E2M1, NC_E5M2>(p, t, stream);
}

}  // namespace nc
