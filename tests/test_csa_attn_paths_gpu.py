"""fm_csa_attn / fm_csa_attn_tree on the ways that a call can take: whole items,
clusters that join their splits, and partial results through memory.  Which one a
call took shows in its workspace: only the last writes there."""
import numpy as np
import pytest

import attn_ref as ref
from test_csa_attn_gpu import Batch, torch_dev  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
D, PAGE = ref.D, ref.PAGE


def shifted(torch, t, elements):
    """The tensor's copy, `elements` behind the start of an allocation."""
    big = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    view = big[elements:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("seqs,window", [([(1, 2600)], 2601), ([(30, 300)], 150), ([(200, 230)], 100)])
def test_arguments_on_their_own_borders_only(torch_dev, seqs, window, tree):
    """Positions and tree bases on an 8-byte border and no wider one, 32-bit arguments
    on a 4-byte one, with keys that are none in every tile that can have them."""
    torch, dev = torch_dev
    b = Batch(1200 + window, seqs, 20, 70, window, 3, holes=True, pads=2, tree=tree)
    b.device(torch, dev)
    for args, names in ((b.d, ("page_table", "pos")), (b.kw, ("seq", "cells", "sink_logit", "lse_out", "tree_mask", "tree_base"))):
        for name in names:
            if args.get(name) is not None:
                args[name] = shifted(torch, args[name], 1)
                assert args[name].data_ptr() % (2 * args[name].element_size()) != 0
    b.call()
    b.check(torch)
