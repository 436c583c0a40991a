// attn_f16_96.hip -- the kernels of attn.hpp for one type of input and one width of the contracted side.
#include "attn.hpp"

namespace gsr {
GSR_ATTN_KERNELS(_Float16, 96)
}  // namespace gsr
