"""MI355X-native Muon optimizer step: a C-ABI HIP library (libmuon.so, include/muon.h)
with a thin PyTorch binding.

    from orthogonalized_momentum_optimizer_amd import Muon
    opt = Muon(model_matrices, lr=0.02, momentum=0.95, nesterov=True, ns_steps=5)
    adam = CautiousAdam(other_params, lr=1e-3, betas=(0.9, 0.999), weight_decay=0.01)
    clip_grad_norm_(all_params, max_norm=1.0)

or, for all parameters at once, with 8-bit states and clipping inside the step:

    from orthogonalized_momentum_optimizer_amd import AdamW
    opt = AdamW(params, lr=6e-4, weight_decay=0.1, state_bits=8, max_grad_norm=1.0)

and for the products of a model whose weights Muon steps, in microscaled 4-bit values:

    copies = MX4Copies(model_matrices)
    opt = Muon(model_matrices, lr=0.02, mx4_copies=copies)
    y = mx4_linear(x, w, copies[w])

``orthogonalize`` runs the Newton-Schulz rounds on stacks of small matrices (attention heads).

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
from .mx4 import (  # noqa: F401
    MX4Copies,
    MX4Tensor,
    mx4_linear,
    mx4_matmul,
    mx4_quantize,
    mx4_quantize_both,
)
from .optim import (  # noqa: F401
    CautiousAdam,
    Muon,
    MuonPlan,
    cautious_adam_step,
    make_adam_config,
    make_config,
    orthogonalize,
    zeropower_via_newtonschulz5,
)
