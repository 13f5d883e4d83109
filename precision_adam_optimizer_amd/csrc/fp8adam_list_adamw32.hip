// fp8adam_list_adamw32.hip -- instantiates the list AdamW kernels with 32-bit moments.
#include "fp8adam_list.h"

namespace fp8adam_list {

template int launch_adamw<false, 0, 0>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&, int64_t,
                                       const AdamwCtl*, hipStream_t);

}  // namespace fp8adam_list
