// device.hpp -- what every host entry point asks of the current device.
#pragma once

namespace gbt {

// GEMM_BT_OK and the compute-unit count when the current device is a gfx950
// (looked up once per device), else GEMM_BT_ERR_NO_DEVICE.
int check_device(int* num_cu);

// The count that plans are made for: the current device's, or 256 without one.
int plan_cus();

}  // namespace gbt
