// libpasa.so: the C ABI of tree attention on the 4-bit cache (include/pasa.h).
#include "host_util.cuh"

namespace pasa {
int tree_take_device_error(unsigned long long* info) { return take_device_error(info); }
}  // namespace pasa
