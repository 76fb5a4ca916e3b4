// Shared-prefix attention parts for head dimension d = 128.
#include "launch_prefix_tiles.cuh"

template int srftq::launch_prefix_tiles<128>(const srftq::PrefixArgs&, int, int, cudaStream_t);
