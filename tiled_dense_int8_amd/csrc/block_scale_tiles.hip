// Instantiates the LDS tile kernels of the block-scaled e4m3 product.
#include "block_scale_kernel.h"
#include "product_table.h"

namespace tdi8 {

void register_f8_tiles(const void **k) {
    k[0] = reinterpret_cast<const void *>(&block_scale_kernel<F8, 1, 4, 4, 2, 4>);
    k[1] = reinterpret_cast<const void *>(&block_scale_kernel<F8, 2, 2, 4, 4, 4>);
    k[2] = reinterpret_cast<const void *>(&block_scale_kernel<F8, 2, 2, 4, 4, 2>);
    k[3] = reinterpret_cast<const void *>(&block_scale_kernel<F8, 2, 4, 8, 4, 2>);
}
void register_f8wide_tiles(const void **k) {
    k[0] = reinterpret_cast<const void *>(&block_scale_kernel<F8Wide, 1, 4, 4, 2, 4>);
    k[1] = reinterpret_cast<const void *>(&block_scale_kernel<F8Wide, 2, 2, 4, 4, 4>);
    k[2] = reinterpret_cast<const void *>(&block_scale_kernel<F8Wide, 2, 2, 4, 4, 2>);
}

}  // namespace tdi8
