// Cache writes in the INT4 codebook (see kv_rows.h).
#include "kv_rows.h"

namespace ufp4 {

hipError_t kv_write_int4(const KvRows& p, hipStream_t s) { return kv::write_grid<1>(p, s); }

}  // namespace ufp4
