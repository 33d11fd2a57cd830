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


MARK = 0xA5


def call_by(torch, b, way):
    """One call, and proof of the way it took.  Whole items and clusters leave the
    workspace as it was; partial results fill exactly [parts, 64] maxima and sums
    and the [parts, 64, 512] outputs behind them."""
    ws = b.kw["workspace"]
    ws.fill_(MARK)
    b.call()
    torch.cuda.synchronize()
    items = b.T * ((b.H + 63) // 64)
    if way != "memory":
        assert items > 128 if way == "whole" else items <= 76
        assert ws.numel() == 0 or bool((ws == MARK).all())
        return
    slots = min(b.window, b.R * PAGE) + min(b.n_sink, b.R * PAGE) + b.k + 32 * b.words
    sms = torch.cuda.get_device_properties(ws.device).multi_processor_count
    splits = min(min(sms, 256) // items, -(-slots // 64))
    parts = items * splits
    assert splits > 1
    assert bool((ws[:parts * 512].view(-1, 8) != MARK).any(1).all())  # a maximum and a sum for each part's 64 heads
    outs = ws[parts * 512:parts * (512 + 64 * 2048)].view(parts, 64, 2048)
    last = b.H - 64 * ((b.H + 63) // 64 - 1)
    assert bool((outs[:, :last] != MARK).any(-1).all())
    assert bool((ws[parts * (512 + 64 * 2048):] == MARK).all())


@pytest.mark.parametrize("H", [2, 33, 64, 80, 130, 320])
@pytest.mark.parametrize("holes", [False, True])
def test_through_memory(torch_dev, H, holes):
    """Partial results of one to five blocks of heads, the last one full and not, of a
    long token and of one that leaves most of its splits without keys; a maximum
    that moves."""
    torch, dev = torch_dev
    seqs = [(1, 7000)] if H > 130 else [(1, 7000), (1, 31)]
    b = Batch(1300 + H, seqs, H, 40, 7001, 2, magnitude=6.0, holes=holes).device(torch, dev)
    call_by(torch, b, "memory")
    b.check(torch)


@pytest.mark.parametrize("H", [5, 64, 80])
@pytest.mark.parametrize("holes", [False, True])
def test_tree_through_memory(torch_dev, H, holes):
    torch, dev = torch_dev
    b = Batch(1400 + H, [(2, 7000)], H, 40, 7001, 2, magnitude=6.0, holes=holes, tree=True).device(torch, dev)
    call_by(torch, b, "memory")
    b.check(torch)


@pytest.mark.parametrize("H", [33, 64, 80])
@pytest.mark.parametrize("tree", [False, True])
def test_output_over_the_queries_through_memory(torch_dev, H, tree):
    torch, dev = torch_dev
    b = Batch(1500 + H, [(2, 7000)], H, 40, 7001, 2, tree=tree).device(torch, dev)
    b.d["out"] = b.d["q"]
    call_by(torch, b, "memory")
    b.check(torch)


COUNTED = [
    # way, tree, seqs, H, k, window, n_sink
    ("whole", False, [(160, 3100)], 20, 30, 2991, 5),
    ("whole", True, [(150, 3100)], 20, 0, 2991, 5),
    ("cluster", False, [(3, 4000), (1, 3333), (1, 12)], 64, 70, 3001, 65),     # of eight
    ("cluster", False, [(30, 3200)], 64, 512, 2500, 4),                        # of four
    ("cluster", False, [(60, 3200)], 20, 512, 600, 4),                         # of two
    ("cluster", True, [(16, 4100)], 64, 33, 3333, 4),
    ("memory", False, [(1, 7000)], 64, 0, 6990, 3),
    ("memory", False, [(2, 6999)], 80, 100, 6500, 66),
    ("memory", True, [(3, 6900)], 64, 10, 6800, 4),
]


@pytest.mark.parametrize("way,tree,seqs,H,k,window,n_sink", COUNTED)
@pytest.mark.parametrize("holes", [False, True])
def test_no_key_is_lost_or_doubled(torch_dev, way, tree, seqs, H, k, window, n_sink, holes):
    """Queries near zero: every key weighs the same, lse is the logarithm of their
    number, good to 2^-18 * (2 + lse) or so, and each key raises one element of the
    output by 1024 / number.  A key more or less at the edge of a window, a page, a
    tile or a split moves lse by 1 / 7000 at least, nearly four times its tolerance, and
    that element by seven times its own."""
    torch, dev = torch_dev
    b = Batch(1600 + H + k, seqs, H, k, window, n_sink, tree=tree, holes=holes, magnitude=2.0 ** -20, sink=False)
    for pool in (b.kv, b.cp):
        used = np.flatnonzero(pool[:, 0] != 0x7FC1)
        pool[used, used * 37 % D] = ref.bf16(np.float32(1024.0))
    b.device(torch, dev)
    call_by(torch, b, way)
    b.check(torch, tokens=None if b.T < 40 else sorted(set(range(0, b.T, 9)) | {b.T - 1}))


def test_tree_with_a_base_past_every_table(torch_dev):
    """Its drafted slots are past the table: no keys, and flagged.  Its committed
    tokens are those of its window, and they are attended to."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    b = Batch(1700, [(4, 100)], 8, 10, 40, 3, tree=True)
    b.rows = []
    for p in b.pos:
        rows = [int(b.table[0, j // PAGE]) * PAGE + j % PAGE for j in ref.visible(p, b.window, b.n_sink, p + 1)]
        b.kv[rows] = ref.bf16(np.random.default_rng(p).standard_normal((len(rows), D)))
        b.rows.append(rows)
    b.device(torch, dev)
    b.kw["tree_base"].fill_(2 ** 63 - 1)
    b.call()
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == fm.FM_DEVERR_PAGE_RANGE
    b.check(torch)


def test_a_layer_without_cached_tokens(torch_dev):
    """Selected cells alone: a pool of no pages and a table of no columns, with
    positions like any other, and nothing flagged."""
    torch, dev = torch_dev
    b = Batch(1800, [(3, 900), (1, 40)], 64, 200, 0, 0).device(torch, dev)
    b.d.update(kv_pool=torch.empty((0, PAGE, D), dtype=torch.int16, device=dev),
               page_table=torch.empty((b.B, 0), dtype=torch.int32, device=dev))
    b.call()
    b.check(torch)


def test_most_heads_and_cells(torch_dev):
    torch, dev = torch_dev
    b = Batch(1900, [(2, 1000)], 1024, 1024, 65, 4).device(torch, dev)
    b.call()
    b.check(torch)


def test_widest_tree(torch_dev):
    """1024 drafted tokens, 32 words of mask."""
    torch, dev = torch_dev
    b = Batch(1901, [(1024, 300)], 20, 8, 64, 4, tree=True)
    assert b.words == 32
    b.device(torch, dev).call()
    b.check(torch, tokens=[0, 1, 31, 32, 33, 500, 1000, 1022, 1023])


@pytest.mark.parametrize("tokens,way", [(1, "memory"), (130, "whole")])
def test_longest_table(torch_dev, tokens, way):
    """The most pages of a table, 2^25 visible tokens, split and not.  All pages are one
    page, and the queries are zero, so every weight is 1 and every partial sum an
    integer that is exact in fp32 up to 2^24: lse is log 2^25, and the output the page's
    mean.  (One element's mean is 1/2: its sums reach 2^24 and pass it by less than 64
    within the last pages, so each of their last steps is off by 1 at most, 2^-19 of
    the mean together.)"""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    R, H = 1 << 19, 3
    g = torch.Generator(device=dev).manual_seed(3)
    page = (torch.randint(0, 2, (1, PAGE, D), generator=g, device=dev) * 2 - 1).bfloat16()
    mean = page[0].double().mean(0)
    assert float(mean.abs().max()) * (1 << 25) <= 1 << 24
    out = torch.empty((tokens, H, D), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((tokens, H), device=dev)
    ws = torch.full((fm.fm_csa_attn_workspace(tokens, H),), MARK, dtype=torch.uint8, device=dev)
    fm.fm_csa_attn(torch.zeros_like(out), page, torch.zeros((1, R), dtype=torch.int32, device=dev),
                   torch.full((tokens,), R * PAGE - 1, device=dev), out, R * PAGE,
                   seq=torch.zeros(tokens, dtype=torch.int32, device=dev), lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    assert (way == "memory") == bool((ws != MARK).any())
    n = 25 * np.log(2.0)
    assert float((lse.double() - n).abs().max()) <= 2.0 ** -18 * (1 + n)
    assert bool(((out.double() - mean).abs() <= ref.HALF_BF16 * mean.abs() * (1 + 2.0 ** -8) + 2.0 ** -16).all())


def test_queries_and_outputs_past_32_bit_offsets(torch_dev):
    """More than 2^32 elements of queries and outputs (8.6 GB each)."""
    torch, dev = torch_dev
    T, H = (1 << 32) // (64 * D) + 30, 64
    b = Batch(1902, [(3, 200)], H, 20, 100, 4).device(torch, dev)
    far = [0, T // 2 + 1, T - 1]  # the batch's three tokens; the others are padding
    q = torch.zeros((T, H, D), dtype=torch.int16, device=dev)
    out, lse = torch.full_like(q, 0x7FC1), torch.full((T, H), float("nan"), device=dev)
    seq, pos = torch.full((T,), -1, dtype=torch.int32, device=dev), torch.zeros(T, dtype=torch.int64, device=dev)
    cells = torch.full((T, 20), -1, dtype=torch.int32, device=dev)
    for i, t in enumerate(far):
        q[t], seq[t], pos[t], cells[t] = b.d["q"][i], 0, b.d["pos"][i], b.kw["cells"][i]
    small = b.d["out"], b.kw["lse_out"]
    b.d.update(q=q, out=out, pos=pos)
    b.kw.update(seq=seq, cells=cells, lse_out=lse, workspace=None)
    b.call()
    torch.cuda.synchronize()
    pad = torch.ones(T, dtype=torch.bool, device=dev)
    pad[far] = False
    assert int((out != 0).any(-1).any(-1).sum()) == 3 and bool(torch.isneginf(lse[pad]).all())
    for i, t in enumerate(far):
        small[0][i], small[1][i] = out[t], lse[t]
    b.d["out"], b.kw["lse_out"] = small
    b.check(torch)
