// Instances of the paged decode kernel: bf16 cache, d = 64, every mode.
#include "paged_decode.cuh"

namespace lssar {
namespace paged {

LSSAR_PAGED_DECODE_INSTANCES(__nv_bfloat16, 64, bf16_d64)

}  // namespace paged
}  // namespace lssar
