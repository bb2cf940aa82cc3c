"""What VocabOps checks before it calls the library, on the host: the calls stop before any kernel."""
import pytest
import torch

import lm_head_vocab_gb300._lib as L
from lm_head_vocab_gb300 import VocabOps


@pytest.fixture(scope="module")
def ops():
    L.build()
    L.load()
    h = VocabOps.__new__(VocabOps)      # no handle: tensors on the host, the library's own checks only
    h.device, h._index, h.handle, h.workspace_bytes = torch.device("cpu"), -1, None, 0
    return h


def test_views_that_stand_for_other_values_are_refused(ops):
    # a conjugated or negated view holds the bytes of what it was made from
    x = torch.randn(6, 4, dtype=torch.complex64)
    plain = torch.empty(6, 4, dtype=torch.complex64)
    for t, o in ((x.conj(), plain), (plain, x.conj()), (x.conj().imag, torch.empty(6, 4)), (x.real, x.conj().imag)):
        assert t.is_conj() or t.is_neg() or o.is_conj() or o.is_neg()
        with pytest.raises(ValueError, match="conjugate"):
            ops._describe(t, o, 0, 6, 6)
    ops._describe(x.conj(), x.conj(), 0, 6, 6)                   # moved as they are
    ops._describe(x, plain, 0, 6, 6)
    with pytest.raises(ValueError, match="conjugate"):
        ops.embedding_forward(torch.view_as_complex(torch.randn(6, 4, 2)).conj().imag, torch.zeros(3, dtype=torch.int64))
