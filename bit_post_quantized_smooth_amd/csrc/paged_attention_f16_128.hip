// The attention over a paged cache for heads of up to 128 fp16 channels.
#include "paged_attention_kernel.hpp"

namespace svdq {

template void launch_paged_tiles<_Float16, 128>(const PagedArgs&, unsigned, hipStream_t);

}  // namespace svdq
