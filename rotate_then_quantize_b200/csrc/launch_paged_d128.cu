// Paged codec for head dimension d = 128.
#include "launch_paged.cuh"

template int srftq::launch_quantize_paged<128>(const srftq::PagedCall&);
template int srftq::launch_dequantize_paged<128>(const srftq::PagedCall&);
