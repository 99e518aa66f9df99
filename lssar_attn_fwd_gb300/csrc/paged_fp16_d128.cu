// Instances of the paged decode kernel: fp16 cache, d = 128, every mode.
#include "paged_decode.cuh"

namespace lssar {
namespace paged {

LSSAR_PAGED_DECODE_INSTANCES(__half, 128, fp16_d128)

}  // namespace paged
}  // namespace lssar
