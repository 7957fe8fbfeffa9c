// The windowed attention kernels for one (K format, V format) pair, chosen at
// compile time with -DPA_KT=<pa_type> -DPA_VT=<pa_type>; compiled once per pair.
#include "pa_step_impl.cuh"
#include "pa_window_impl.cuh"

#if !defined(PA_KT) || !defined(PA_VT)
#error "compile with -DPA_KT=<pa_type> -DPA_VT=<pa_type>"
#endif

#define PA_WINDOW_NAME_(k, v) lookup_window_kernel_##k##_##v
#define PA_WINDOW_NAME(k, v) PA_WINDOW_NAME_(k, v)
#define PA_STEP_NAME_(k, v) lookup_step_kernel_##k##_##v
#define PA_STEP_NAME(k, v) PA_STEP_NAME_(k, v)

namespace pa_prefix {

bool PA_WINDOW_NAME(PA_KT, PA_VT)(WindowKernel* out) {
  *out = WindowKernel{pa_prefix_kernel<PA_KT, PA_VT, WindowParams>, Smem<PA_KT, PA_VT, true>::kLaunch};
  return true;
}

bool PA_STEP_NAME(PA_KT, PA_VT)(StepKernel* out) {
#if PA_KT == 8 && PA_VT != 1
  *out = StepKernel{pa_step_kernel<PA_VT>, StepSmem<PA_VT>::kTotal};
#else
  *out = StepKernel{nullptr, 0};
#endif
  return true;
}

}  // namespace pa_prefix
