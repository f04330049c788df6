// entry.h -- the forward pass behind the extern "C" entry points and the device
// check, for the entry points defined outside api.cpp.
#pragma once

#include "mdcn.h"

namespace mdcn {

// mdcn_forward's work (validation, planning, launches on `stream`) with the
// given workspace; the same contract and status codes.
mdcn_status forward_with_workspace(const mdcn_op *op, mdcn_dtype dtype, const int64_t dims[16],
                                   const void *x, const void *offset, const void *mask,
                                   const void *weight, const void *bias, int64_t bias_len,
                                   void *out, void *workspace, size_t workspace_bytes,
                                   void *stream);

// MDCN_OK if the current device is a gfx950 GPU, else MDCN_E_DEVICE.
mdcn_status check_device();

}  // namespace mdcn
