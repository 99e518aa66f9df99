// Instances of the paged decode kernel: fp16 cache, d = 64, every mode.
#include "paged_decode.cuh"

namespace lssar {
namespace paged {

LSSAR_PAGED_DECODE_INSTANCES(__half, 64, fp16_d64)

}  // namespace paged
}  // namespace lssar
