// Shared-prefix attention parts for head dimension d = 64.
#include "launch_prefix_tiles.cuh"

template int srftq::launch_prefix_tiles<64>(const srftq::PrefixArgs&, int, int, cudaStream_t);
