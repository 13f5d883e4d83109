// fp8adam_layer_grad_e4m3.hip -- instantiates the products of the backward pass with codes in E4M3.
#include "fp8adam_layer_grad.h"

namespace fp8adam_layer {

template int launch_grad<0>(const GradArgs&, const GradPlan&, hipStream_t);

}  // namespace fp8adam_layer
