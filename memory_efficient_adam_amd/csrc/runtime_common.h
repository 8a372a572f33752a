// What the host runtimes of one library share: the calling thread's last
// error, and what a step's arguments mean.
#pragma once

#include <string>

#include "adam_internal.h"
#include "adam_mi355x.h"

namespace adam_mi355x {

// Records msg as the calling thread's last error (adam_last_error) and
// returns code.
int set_last_error(int code, const std::string &msg);

// A step's checks of its layout and hyperparameters (an adam_status), and the
// kernel's scalars from the latter.
int check_adam_layout(const adam_layout *l);
int check_adam_hparams(const adam_hparams *hp, int32_t storage);
void adam_scalars(StepArgs &a, const adam_hparams *hp);

}  // namespace adam_mi355x
