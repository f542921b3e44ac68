// vdit_internal.h - what the library's translation units share on the host side.
#pragma once

namespace vdit {

// Device address, on the current device, of the watchdog's flag word, or null
// if the runtime reports an error.  The flag is one device symbol of
// vdit_api.cu; kernels of other translation units take its address as an
// argument.
const unsigned int* watchdog_flag();

// 128-token blocks of a sequence.
inline int sparse_blocks(int L) { return (int)(((long long)L + 127) / 128); }

}  // namespace vdit
