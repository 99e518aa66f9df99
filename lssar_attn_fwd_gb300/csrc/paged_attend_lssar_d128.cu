// Instances of the chunk attention: lssar, d = 128, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(lssar_d128, kLssar, 128)

}  // namespace attend
}  // namespace lssar
