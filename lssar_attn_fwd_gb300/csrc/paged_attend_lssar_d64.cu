// Instances of the chunk attention: lssar, d = 64, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(lssar_d64, kLssar, 64)

}  // namespace attend
}  // namespace lssar
