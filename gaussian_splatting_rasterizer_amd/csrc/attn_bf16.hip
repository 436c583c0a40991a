// attn_bf16.hip -- the kernels of attn.hpp for one type of input.
#include "attn.hpp"

namespace gsr {
GSR_ATTN_KERNELS(__bf16)
}  // namespace gsr
