// The attention kernels of several causal new tokens.
#include "fa_decode_select.cuh"

namespace fa {

DecodeKernel decode_kernel_partly(int d, bool f8, const DecodeLayout &l) { return decode_kernel<true>(d, f8, l); }

}  // namespace fa
