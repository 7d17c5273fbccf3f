// dan_rows_lnsave.cu -- launches of the LayerNorm + modulate row kernel that
// keeps what the gradient needs (include/dan_train.h).
#include "dan_rows.cuh"

namespace dan {

cudaError_t launch_ln_modulate_save(const RowProblem &q, cudaStream_t s)
{
    return (q.D % 1024) ? launch_ln_fpt<kLnSave, true>(q, s) : launch_ln_fpt<kLnSave, false>(q, s);
}

} // namespace dan
