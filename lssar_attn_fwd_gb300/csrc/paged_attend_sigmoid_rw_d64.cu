// Instances of the chunk attention: sigmoid_rw, d = 64, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(sigmoid_rw_d64, kSigmoidRw, 64)

}  // namespace attend
}  // namespace lssar
