// The order of a call's launches among those of other host threads.
#pragma once

#include <mutex>

namespace pa {

// Held while the kernels of a call on this workspace are queued. Host threads that call on one
// stream share its workspace: with a launch of another's between the two of a call, its second
// kernel would join what the other's first one left. (Workspaces may share a mutex.)
std::mutex& launch_mutex(const void* workspace);

}  // namespace pa
