// Instances of the chunk attention: lssa, d = 64, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(lssa_d64, kLssa, 64)

}  // namespace attend
}  // namespace lssar
