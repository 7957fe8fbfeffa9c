// The shared-prefix decode kernel for one (K format, V format) pair, chosen at
// compile time with -DPA_KT=<pa_type> -DPA_VT=<pa_type>; compiled once per pair.
#include "pa_prefix_impl.cuh"

#if !defined(PA_KT) || !defined(PA_VT)
#error "compile with -DPA_KT=<pa_type> -DPA_VT=<pa_type>"
#endif

#define PA_PREFIX_NAME_(k, v) lookup_prefix_kernel_##k##_##v
#define PA_PREFIX_NAME(k, v) PA_PREFIX_NAME_(k, v)

namespace pa_prefix {

bool PA_PREFIX_NAME(PA_KT, PA_VT)(KernelInfo* out) {
  *out = KernelInfo{pa_prefix_kernel<PA_KT, PA_VT>, Smem<PA_KT, PA_VT>::kLaunch};
  return true;
}

}  // namespace pa_prefix
