// The windowed attention kernel for one (K format, V format) pair, chosen at
// compile time with -DPA_KT=<pa_type> -DPA_VT=<pa_type>; compiled once per pair.
#include "pa_window_impl.cuh"

#if !defined(PA_KT) || !defined(PA_VT)
#error "compile with -DPA_KT=<pa_type> -DPA_VT=<pa_type>"
#endif

#define PA_WINDOW_NAME_(k, v) lookup_window_kernel_##k##_##v
#define PA_WINDOW_NAME(k, v) PA_WINDOW_NAME_(k, v)

namespace pa_prefix {

bool PA_WINDOW_NAME(PA_KT, PA_VT)(WindowKernel* out) {
  *out = WindowKernel{pa_prefix_kernel<PA_KT, PA_VT, WindowParams>, Smem<PA_KT, PA_VT, true>::kLaunch};
  return true;
}

}  // namespace pa_prefix
