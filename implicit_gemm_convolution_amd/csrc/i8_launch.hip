// i8_launch.hip -- the kernels of the products in 8 bits: launch_product of
// ffn_host.hpp for the pairs of IGC_I8_KINDS.  The build compiles this file once
// for each with -DIGC_I8_UNIT=<n>.
#include "product_launch.hpp"

namespace igc_ffn_host {

#define IGC_I8_DEFINE(BF, MODE) template int launch_product<BF, MODE>(const igc_ffn::GemmArgs&, const Plan&, hipStream_t);
#if IGC_I8_UNIT == 0
IGC_I8_DEFINE(false, igc_ffn::M_I8)
#elif IGC_I8_UNIT == 1
IGC_I8_DEFINE(true, igc_ffn::M_I8)
#elif IGC_I8_UNIT == 2
IGC_I8_DEFINE(false, igc_ffn::M_I8_GLU)
#elif IGC_I8_UNIT == 3
IGC_I8_DEFINE(true, igc_ffn::M_I8_GLU)
#else
#error "IGC_I8_UNIT: 0 .. 3"
#endif

}  // namespace igc_ffn_host
