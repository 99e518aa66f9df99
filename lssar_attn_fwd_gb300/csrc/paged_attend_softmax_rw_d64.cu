// Instances of the chunk attention: softmax_rw, d = 64, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(softmax_rw_d64, kSoftmaxRw, 64)

}  // namespace attend
}  // namespace lssar
