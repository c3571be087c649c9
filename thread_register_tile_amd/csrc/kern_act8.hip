// kern_act8.hip -- instances of the 8-bit activations' row kernels.
#include "act8.hpp"
#include "launch.hpp"

namespace trt {

namespace {

template <class F>
hipError_t with_type(int dt, F&& f) {
  if (dt == DT_F16) return f.template operator()<DT_F16>();
  if (dt == DT_BF16) return f.template operator()<DT_BF16>();
  return f.template operator()<DT_F32>();
}

}  // namespace

hipError_t launch_act8_pack(const Act8Args& a, int dt, int64_t groups, hipStream_t s) {
  return with_type(dt, [&]<int DT>() { return launch(act8_pack_kernel<DT>, dim3(groups), dim3(256), 0, s, a); });
}

hipError_t launch_act8_unpack(const Act8Args& a, int dt, int64_t groups, hipStream_t s) {
  return with_type(dt, [&]<int DT>() { return launch(act8_unpack_kernel<DT>, dim3(groups), dim3(256), 0, s, a); });
}

hipError_t launch_act8_operands(const Act8OperandArgs& a, int dt, int64_t groups, hipStream_t s) {
  if (dt == DT_F16) return launch(act8_operands_kernel<DT_F16>, dim3(groups), dim3(256), 0, s, a);
  return launch(act8_operands_kernel<DT_BF16>, dim3(groups), dim3(256), 0, s, a);
}

hipError_t launch_act8_sum(const Act8SumArgs& a, int odt, hipStream_t s) {
  const int64_t groups = ((int64_t)a.rows * (a.part_ld / 4) + 255) / 256;
  return with_type(odt, [&]<int OT>() {
    return launch(act8_sum_kernel<OT>, dim3(groups < (1 << 20) ? groups : 1 << 20), dim3(256), 0, s, a);
  });
}

}  // namespace trt
