// Cache writes in the E1M2 codebook (see kv_rows.h).
#include "kv_rows.h"

namespace ufp4 {

hipError_t kv_write_e1m2(const KvRows& p, hipStream_t s) { return kv::write_grid<0>(p, s); }

}  // namespace ufp4
