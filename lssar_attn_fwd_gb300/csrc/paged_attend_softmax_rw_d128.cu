// Instances of the chunk attention: softmax_rw, d = 128, both types.
#include "paged_attend.cuh"

namespace lssar {
namespace attend {

LSSAR_ATTEND_INSTANCE(softmax_rw_d128, kSoftmaxRw, 128)

}  // namespace attend
}  // namespace lssar
