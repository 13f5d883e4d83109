// fp8adam_list_adamw8_e4m3_e4m3.hip -- instantiates the list AdamW kernels with 8-bit moments, m in E4M3
// and v in E4M3 (one translation unit per format pair, so the library builds in parallel).
#include "fp8adam_list.h"

namespace fp8adam_list {

template int launch_adamw<true, 0, 0>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&, int64_t,
                                        const AdamwCtl*, hipStream_t);

}  // namespace fp8adam_list
