// Many-adapter block-circulant kernels for block size p = 4096 (one translation unit per p).
#include "circ_many.cuh"

namespace rdfft {
RDFFT_CIRC_MANY_INSTANCE(4096)
}  // namespace rdfft
