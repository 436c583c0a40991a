// attn_f32_64.hip -- the kernels of attn.hpp for one type of input and one width of the contracted side.
#include "attn.hpp"

namespace gsr {
GSR_ATTN_KERNELS(float, 64)
}  // namespace gsr
