// cross.cu -- rows that see all of another sequence (an encoder's states): the forms of window.cuh
// with every row's view the same, so that only a sequence's last tile has columns to hide.
#include "window.cuh"

namespace sfi {

cudaError_t launch_cross(const WindowParams &p, int rows, bool shares, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                         const CUtensorMap &tm_q, int grid, cudaStream_t stream)
{
    return launch_rows<true>(p, rows, shares, tm_k, tm_v, tm_q, grid, stream);
}

}  // namespace sfi
