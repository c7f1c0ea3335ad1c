#include "nc_kv_few.h"

namespace nc {
hipError_t kv_few_e4m3_bf16(const KvAttn& a, int dim, const KvPlan& p, hipStream_t s) { return few_by_dim<NC_E4M3, NC_BF16>(a, dim, p, s); }
}  // namespace nc
