// Products with many rows whose first operand is E4M3.
#include "nc_mx_many.h"

namespace nc {

hipError_t mx_many_e4m3(const MxProduct& p, int fb, int w, hipStream_t stream) {
  return fb == NC_E2M1 ? mx_many_launch<NC_E4M3, NC_E2M1>(p, w, stream)
       : fb == NC_E4M3 ? mx_many_launch<NC_E4M3, NC_E4M3>(p, w, stream)
                       : mx_many_launch<NC_E4M3, NC_E5M2>(p, w, stream);
}

}  // namespace nc
