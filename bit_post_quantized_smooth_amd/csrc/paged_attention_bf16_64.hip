// The attention over a paged cache for heads of up to 64 bf16 channels.
#include "paged_attention_kernel.hpp"

namespace svdq {

template void launch_paged_tiles<__bf16, 64>(const PagedArgs&, unsigned, hipStream_t);

}  // namespace svdq
