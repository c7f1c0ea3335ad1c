#include "nc_kv_many.h"

namespace nc {
hipError_t kv_many_e4m3_bf16(const KvAttn& a, int dim, hipStream_t s) { return many_by_dim<NC_E4M3, NC_BF16>(a, dim, s); }
}  // namespace nc
