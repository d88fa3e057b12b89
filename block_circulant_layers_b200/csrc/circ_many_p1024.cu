// Many-adapter block-circulant kernels for block size p = 1024 (one translation unit per p).
#include "circ_many.cuh"

namespace rdfft {
RDFFT_CIRC_MANY_INSTANCE(1024)
}  // namespace rdfft
