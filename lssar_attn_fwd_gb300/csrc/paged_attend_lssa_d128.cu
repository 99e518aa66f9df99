// Instances of the chunk attention: lssa, d = 128, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(lssa_d128, kLssa, 128)

}  // namespace attend
}  // namespace lssar
