// Cache writes in the E2M1 codebook (see kv_rows.h).
#include "kv_rows.h"

namespace ufp4 {

hipError_t kv_write_e2m1(const KvRows& p, hipStream_t s) { return kv::write_grid<2>(p, s); }

}  // namespace ufp4
