// Many-adapter block-circulant kernels for block size p = 128 (one translation unit per p).
#include "circ_many.cuh"

namespace rdfft {
RDFFT_CIRC_MANY_INSTANCE(128)
}  // namespace rdfft
