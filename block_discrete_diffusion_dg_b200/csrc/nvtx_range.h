// Profiler ranges of the entry points.
#pragma once

#include <nvtx3/nvToolsExt.h>

namespace dg {

// NVTX range over one entry point's host work (its checks and launches); a profiler projects it
// onto the kernels it launched, so a timeline groups them under the call (and the layer) that
// issued them.  Without an attached tool the calls return at once.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  // a range named `name` carrying an integer payload (the layer index)
  NvtxRange(const char *name, int payload) {
    nvtxEventAttributes_t a{};
    a.version = NVTX_VERSION;
    a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
    a.messageType = NVTX_MESSAGE_TYPE_ASCII;
    a.message.ascii = name;
    a.payloadType = NVTX_PAYLOAD_TYPE_INT32;
    a.payload.iValue = payload;
    nvtxRangePushEx(&a);
  }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

}  // namespace dg
