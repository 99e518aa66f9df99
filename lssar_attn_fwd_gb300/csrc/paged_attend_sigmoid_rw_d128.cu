// Instances of the chunk attention: sigmoid_rw, d = 128, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(sigmoid_rw_d128, kSigmoidRw, 128)

}  // namespace attend
}  // namespace lssar
