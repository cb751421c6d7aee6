// The norms around a block whose normed row leaves in 8 bits with group scales,
// staged for the expert layer, beside or instead of the 16-bit one: the layer's
// own staging would read that row again.  Bound by HBM: 16381 x 7168 bf16, y added, codes
// and fp32 scales, no 16-bit copy: 143 us, 826 MB at 5.8 TB/s; 32 x 7168 in 6 us.
#include "norm_forward.h"

namespace moe {

hipError_t launch_norm_quant(const NormArgs& a, int dtype, bool w32, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  switch (dtype) {
    case kBf16:
      return w32 ? norm_dt<kBf16, true, true>(a, stream) : norm_dt<kBf16, false, true>(a, stream);
    case kF16:
      return w32 ? norm_dt<kF16, true, true>(a, stream) : norm_dt<kF16, false, true>(a, stream);
    default: return norm_dt<kF32, true, true>(a, stream);
  }
}

}  // namespace moe
