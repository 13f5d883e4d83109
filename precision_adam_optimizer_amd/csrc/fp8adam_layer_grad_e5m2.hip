// fp8adam_layer_grad_e5m2.hip -- instantiates the products of the backward pass with codes in E5M2.
#include "fp8adam_layer_grad.h"

namespace fp8adam_layer {

template int launch_grad<1>(const GradArgs&, const GradPlan&, hipStream_t);

}  // namespace fp8adam_layer
