// Host helpers of the paged key / value cache shared by the ABI files.
#pragma once
#include "../../include/rdt.h"
#include "kernels.h"

namespace rdt {
rdt_status check_paged_cache(const rdt_paged_cache* c);
PagedView paged_view(const rdt_paged_cache* c, int loop);   // the pages of one loop
}  // namespace rdt
