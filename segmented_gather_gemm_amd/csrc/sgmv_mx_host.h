// sgmv_mx_host.h -- host-side helpers of the entry points that take microscaled
// 4-bit rows.  Internal to libsgmv.
#pragma once

#include "sgmv_host.h"

namespace sgmv {
namespace host {

// Whether `q` holds rows of `cols` values, aligned as the kernels read them.
sgmv_status check_mx(const sgmv_mx_stack& q, int64_t cols, const char* what);

}  // namespace host
}  // namespace sgmv
