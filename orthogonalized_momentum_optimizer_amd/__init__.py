"""MI355X-native Muon optimizer step: a C-ABI HIP library (libmuon.so, include/muon.h)
with a thin PyTorch binding.

    from orthogonalized_momentum_optimizer_amd import Muon
    opt = Muon(model_matrices, lr=0.02, momentum=0.95, nesterov=True, ns_steps=5)
    adam = CautiousAdam(other_params, lr=1e-3, betas=(0.9, 0.999), weight_decay=0.01)
    clip_grad_norm_(all_params, max_norm=1.0)

or, for all parameters at once, with 8-bit states and clipping inside the step:

    from orthogonalized_momentum_optimizer_amd import AdamW
    opt = AdamW(params, lr=6e-4, weight_decay=0.1, state_bits=8, max_grad_norm=1.0)

The library must be built first (``python -m orthogonalized_momentum_optimizer_amd.build``);
importing the optimizer never falls back to another implementation.
"""
from ._lib import MuonError  # noqa: F401
from .adamw import (  # noqa: F401
    AdamW,
    AdamWPlan,
    GradNormPlan,
    clip_grad_norm_,
    grad_norm,
    make_adamw_config,
)
from .optim import (  # noqa: F401
    CautiousAdam,
    Muon,
    MuonPlan,
    cautious_adam_step,
    make_adam_config,
    make_config,
    zeropower_via_newtonschulz5,
)
