// Paged codec for head dimension d = 256.
#include "launch_paged.cuh"

template int srftq::launch_quantize_paged<256>(const srftq::PagedCall&);
template int srftq::launch_dequantize_paged<256>(const srftq::PagedCall&);
