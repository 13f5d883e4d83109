// fp8adam_layer_product_e5m2_e5m2.hip -- instantiates the forward products of inputs in E5M2 and weights in
// E5M2 (one translation unit per format pair, so the library builds in parallel).
#include "fp8adam_layer_product.h"

namespace fp8adam_layer {

template int launch_product<1, 1>(const ProductArgs&, bool, hipStream_t);

}  // namespace fp8adam_layer
