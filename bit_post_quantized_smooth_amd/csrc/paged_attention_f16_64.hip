// The attention over a paged cache for heads of up to 64 fp16 channels.
#include "paged_attention_kernel.hpp"

namespace svdq {

template void launch_paged_tiles<_Float16, 64>(const PagedArgs&, unsigned, hipStream_t);

}  // namespace svdq
