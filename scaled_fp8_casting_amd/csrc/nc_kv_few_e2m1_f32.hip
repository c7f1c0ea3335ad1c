#include "nc_kv_few.h"

namespace nc {
hipError_t kv_few_e2m1_f32(const KvAttn& a, int dim, const KvPlan& p, hipStream_t s) { return few_by_dim<NC_E2M1, NC_F32>(a, dim, p, s); }
}  // namespace nc
