// Many-adapter block-circulant kernels for block size p = 2048 (one translation unit per p).
#include "circ_many.cuh"

namespace rdfft {
RDFFT_CIRC_MANY_INSTANCE(2048)
}  // namespace rdfft
