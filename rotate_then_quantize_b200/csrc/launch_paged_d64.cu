// Paged codec for head dimension d = 64.
#include "launch_paged.cuh"

template int srftq::launch_quantize_paged<64>(const srftq::PagedCall&);
template int srftq::launch_dequantize_paged<64>(const srftq::PagedCall&);
