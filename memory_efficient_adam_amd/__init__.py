"""MI355X-native compressed-moment Adam/AdamW step, and the Muon step with its
Newton-Schulz orthogonalisation for 2-D weights.

Thin Python binding over ``libadam_mi355x.so`` (C ABI in
``include/adam_mi355x.h`` and ``include/muon_mi355x.h``): the functions below carry the C names and only
marshal arguments (torch tensors -> device pointers, the caller's current
HIP stream).  Every step of the update runs in the library's HIP kernels;
there is no CPU or PyTorch fallback -- if the library is not built, the
first call raises.
"""
from ._binding import (  # noqa: F401
    ADAM_BLOCK_SIZE,
    AdamError,
    AdamState,
    BUFFERS,
    GRAD_DTYPES,
    OPT_AMSGRAD,
    STORAGES,
    adam_last_error,
    adam_state_buffer_bytes,
    adam_state_bytes,
    adam_state_create,
    adam_state_describe,
    adam_state_destroy,
    adam_state_get_draw_index,
    adam_state_load,
    adam_state_read,
    adam_state_save,
    adam_state_serialized_bytes,
    adam_state_set_draw_index,
    adam_state_write,
    adam_step,
    adam_step_noalloc,
    library,
    library_path,
    state_buffer_sizes,
)
from ._muon import (  # noqa: F401
    MUON_SCALES,
    MUON_STORAGES,
    MuonState,
    muon_orthogonalize,
    muon_orthogonalize_workspace_bytes,
    muon_state_buffer_bytes,
    muon_state_bytes,
    muon_state_create,
    muon_state_describe,
    muon_state_destroy,
    muon_state_get_draw_index,
    muon_state_load,
    muon_state_momentum,
    muon_state_read,
    muon_state_save,
    muon_state_serialized_bytes,
    muon_state_set_draw_index,
    muon_state_workspace_bytes,
    muon_state_write,
    muon_step,
)
