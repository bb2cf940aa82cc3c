"""lmloss for GB300: fused LM-head loss (collapse-free CE, z-loss, distillation
KL, GSPO) forward + backward over a [T, V] logit matrix, and the operators at the
two ends of the vocabulary (embedding lookup and gradient, beam search's step
and state reordering, token log-probabilities, 4-bit tables), in hand-written sm_103a CUDA behind a C ABI
(include/lmloss.h)."""
from ._lib import LMLossError, build, load  # noqa: F401
from .lmloss import LMLoss, Outputs, lmloss_forward_backward  # noqa: F401
from .vocab import BeamStep, Table4, TokenLogprobs, VocabOps  # noqa: F401
