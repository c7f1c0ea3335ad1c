#include "nc_kv_many.h"

namespace nc {
hipError_t kv_many_e2m1_f32(const KvAttn& a, int dim, hipStream_t s) { return many_by_dim<NC_E2M1, NC_F32>(a, dim, s); }
}  // namespace nc
