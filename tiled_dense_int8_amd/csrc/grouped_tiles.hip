// Instantiates the LDS tile kernels of the int8 product grouped by expert.
#include "product_table.h"
#include "tiled_kernel.h"
#include "rc_pipelined_kernel.h"

namespace tdi8 {

void register_grouped_tiles(const void **k) {
    k[0] = reinterpret_cast<const void *>(&grouped_pipelined_kernel<32, 2, 4, 1, 1, 128, 3>);
    k[1] = reinterpret_cast<const void *>(&grouped_pipelined_kernel<32, 2, 4, 2, 2, 128, 3>);
    k[2] = reinterpret_cast<const void *>(&grouped_pipelined_kernel<32, 2, 4, 4, 2, 128, 2>);
}

}  // namespace tdi8
