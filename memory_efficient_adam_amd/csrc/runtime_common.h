// What the host runtimes of one library share: the calling thread's last
// error.
#pragma once

#include <string>

namespace adam_mi355x {

// Records msg as the calling thread's last error (adam_last_error) and
// returns code.
int set_last_error(int code, const std::string &msg);

}  // namespace adam_mi355x
