// f8_front_kernel for a factor whose rows run along the contraction, V = dY B.  (Compiled
// apart: beside these the other form's code came out 2 to 7% slower.)
#include "f8_front.cuh"

namespace qlora {

const void* front_along_kernel(bool e5m2, bool two) { return front_kernel<true>(e5m2, two); }

}  // namespace qlora
