"""fm_csa_attn / fm_csa_attn_tree against the fp64 formulas, at the sizes, masks
and layouts where they can go wrong.  Every pool row that is no key of any token
is NaN, so a read of it shows."""
import numpy as np
import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu
D, PAGE = ref.D, ref.PAGE


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


class Batch:
    """A ragged batch: seqs = [(new tokens, last position)], each with its pages."""

    def __init__(self, seed, seqs, H, k, window, n_sink, Pc=24, sink=True, holes=False, pads=0, tree=False, gap=1,
                 magnitude=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.k, self.window, self.n_sink, self.tree, self.gap = H, k, window, n_sink, tree, gap
        self.seq, self.pos, masks, base = [], [], [], []
        for b, (n, last) in enumerate(seqs):
            base.append(last + 1)
            if tree:
                anc, depth = [], []
                for i in range(n):
                    par = i - 1 - int(rng.integers(0, 4))
                    anc.append((anc[par] if par >= 0 else 0) | (1 << i))
                    depth.append(depth[par] + 1 if par >= 0 else 1)
                masks += anc
                self.pos += [last + x for x in depth]
            else:
                self.pos += list(range(last - n + 1, last + 1))
            self.seq += [b] * n
        for i in range(pads):  # padding rows behind the batch
            self.seq.append(-1 if i % 2 else 0)
            self.pos.append(-1 if i % 2 == 0 else 5)
            masks.append(0)
        T = self.T = len(self.seq)
        self.words = max(1, (max(n for n, _ in seqs) + 31) // 32) if tree else 0
        self.masks, self.base = masks, base
        B = self.B = len(seqs)
        self.R = max(last + (n if tree else 0) for n, last in seqs) // PAGE + 2
        self.P = B * self.R + 3
        table = rng.permutation(self.P)[:B * self.R].reshape(B, self.R).astype(np.int32)
        if holes:
            table[rng.random(table.shape) < 0.3] = -1
        self.table = table
        self.q = ref.bf16(magnitude * rng.standard_normal((T, H, D)))
        self.sink = rng.standard_normal(H).astype(np.float32) if sink else None
        self.Pc = Pc
        self.cells = np.full((T, k), -1, np.int32)
        for t in range(T):
            n = int(rng.integers(0, k + 1)) if t % 3 else k
            n = min(n, Pc * PAGE)
            c = np.sort(rng.choice(Pc * PAGE, n, replace=False))
            if t % 4 == 3:  # empty entries anywhere, not only at the end
                where = np.sort(rng.choice(k, n, replace=False))
                self.cells[t, where] = c
            else:
                self.cells[t, :n] = c
        # pools: NaN wherever nothing reads
        self.kv = np.full((self.P * PAGE, D), 0x7FC1, np.uint16)
        self.cp = np.full((max(Pc, 1) * PAGE, D), 0x7FC1, np.uint16)
        self.rows = [self.token_rows(t) for t in range(T)]
        used = sorted({r for rows in self.rows for r in rows})
        self.kv[used] = ref.bf16(rng.standard_normal((len(used), D)))
        used = np.unique(self.cells[self.cells >= 0])
        self.cp[used] = ref.bf16(rng.standard_normal((len(used), D)))

    def token_rows(self, t):
        b, p = self.seq[t], self.pos[t]
        if b < 0 or p < 0:
            return []
        slots = ref.visible(p, self.window, self.n_sink, self.base[b] if self.tree else p + 1)
        if self.tree:
            slots += [self.base[b] + i for i in range(32 * self.words) if (self.masks[t] >> i) & 1]
        return [int(self.table[b, j // PAGE]) * PAGE + j % PAGE for j in slots if self.table[b, j // PAGE] >= 0]

    def device(self, torch, dev):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)

        def pool(flat, gap):  # pages with gap - 1 pages of NaN between them
            a = np.full((flat.shape[0] // PAGE, gap, PAGE, D), 0x7FC1, np.uint16)
            a[:, 0] = flat.reshape(-1, PAGE, D)
            return t(a.view(np.int16))[:, 0]
        self.d = dict(q=t(self.q.view(np.int16)), kv_pool=pool(self.kv, self.gap), page_table=t(self.table),
                      pos=t(np.array(self.pos, np.int64)),
                      out=torch.full((self.T, self.H, D), 0x7FC1, dtype=torch.int16, device=dev))
        self.kw = dict(seq=t(np.array(self.seq, np.int32)), window=self.window, n_sink=self.n_sink,
                       sink_logit=None if self.sink is None else t(self.sink),
                       lse_out=torch.full((self.T, self.H), float("nan"), device=dev))
        if self.k:
            self.kw.update(cell_pool=pool(self.cp, self.gap), cells=t(self.cells))
        if self.tree:
            m = np.array([[(x >> (32 * w)) & 0xFFFFFFFF for w in range(self.words)] for x in self.masks], np.uint32)
            self.kw.update(tree_mask=t(m.view(np.int32)), tree_base=t(np.array(self.base, np.int64)))
        import sparse_attention_kv_c4_gb300 as fm
        self.kw["workspace"] = torch.empty(fm.fm_csa_attn_workspace(self.T, self.H), dtype=torch.uint8, device=dev)
        return self

    def call(self):
        import sparse_attention_kv_c4_gb300 as fm
        (fm.fm_csa_attn_tree if self.tree else fm.fm_csa_attn)(**self.d, **self.kw)

    def check(self, torch, tokens=None):
        import sparse_attention_kv_c4_gb300 as fm
        torch.cuda.synchronize()
        assert fm.fm_device_status(reset=True) == 0
        out = ref.f64(self.d["out"].cpu().numpy().view(np.uint16))
        lse = self.kw["lse_out"].cpu().numpy().astype(np.float64)
        for t in range(self.T) if tokens is None else tokens:
            keys = [self.kv[self.rows[t]], self.cp[self.cells[t][self.cells[t] >= 0]]]
            w_out, w_lse, tol, ltol = ref.attend(ref.f64(self.q[t]), ref.f64(np.concatenate(keys)), self.sink, D ** -0.5)
            bad = ~(np.abs(out[t] - w_out) <= tol)
            assert not bad.any(), f"token {t} pos {self.pos[t]} keys {sum(map(len, keys))}: {bad.sum()} values off, " \
                f"first head/element {np.argwhere(bad)[:4].tolist()}, worst {np.nanmax(np.abs(out[t] - w_out)):.3g}"
            both = np.isneginf(w_lse)
            assert (np.isneginf(lse[t]) == both).all(), f"token {t}: lse of a row without keys"
            assert (np.abs(lse[t][~both] - w_lse[~both]) <= ltol[~both]).all(), f"token {t}: lse"


CASES = [
    # seqs, H, k, window, n_sink
    ([(1, 0)], 64, 0, 128, 0),                                   # one token, one key
    ([(1, 36)], 64, 0, 128, 4),
    ([(1, 700)], 1, 1, 1, 0),                                    # one head, one cell, itself
    ([(3, 2), (1, 63), (2, 64), (4, 65)], 20, 37, 63, 1),        # page borders
    ([(5, 129), (1, 0), (7, 400)], 64, 64, 64, 70),              # first tokens beyond a page
    ([(2, 500), (1, 20)], 65, 512, 128, 4),                      # a second head block of one head
    ([(2, 1000)], 128, 1024, 65, 4),                             # the most cells, two head blocks
    ([(1, 5000)], 64, 0, 5001, 0),                               # a long window, split over SMs
    ([(1, 3333), (1, 17)], 130, 100, 3000, 130),
    ([(40, 300)], 64, 130, 0, 0),                                # no tokens at all, cells alone
    ([(40, 300)], 8, 0, 0, 5),                                   # first tokens alone
    ([(333, 332)], 16, 48, 128, 4),                              # a prompt from its first token on
    ([(170, 700), (3, 2)], 64, 72, 130, 3),                      # more tokens than SMs
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("variant", ["plain", "holes"])
def test_matches_formula(torch_dev, case, variant):
    torch, dev = torch_dev
    holes = variant == "holes"
    b = Batch(1000 + case, *CASES[case], holes=holes, pads=3 if holes else 0, sink=not holes, gap=3 if holes else 1)
    b.device(torch, dev).call()
    b.check(torch)


@pytest.mark.parametrize("seqs,H,k,window,n_sink", [
    ([(1, 0)], 64, 0, 128, 0),
    ([(16, 700), (5, 3), (16, 64)], 64, 96, 128, 4),
    ([(61, 900), (33, 62)], 20, 0, 500, 4),
    ([(70, 130)], 128, 40, 1, 0),
    ([(2, 4000)], 64, 0, 100000, 0),
])
@pytest.mark.parametrize("holes", [False, True])
def test_tree_matches_formula(torch_dev, seqs, H, k, window, n_sink, holes):
    torch, dev = torch_dev
    b = Batch(77 + H + k, seqs, H, k, window, n_sink, tree=True, holes=holes, pads=2)
    b.device(torch, dev).call()
    b.check(torch)


@pytest.mark.parametrize("magnitude", [2.0 ** -20, 12.0])
def test_flat_and_sharp_softmax(torch_dev, magnitude):
    """Scores all but equal, and scores that spread over hundreds: the running
    maximum moves from tile to tile."""
    torch, dev = torch_dev
    b = Batch(5, [(9, 900)], 64, 256, 300, 4, magnitude=magnitude)
    b.device(torch, dev).call()
    b.check(torch)


def test_rising_scores(torch_dev):
    """Each key's score is above all before it, by far: every tile moves every
    head's maximum, and all earlier weights vanish."""
    torch, dev = torch_dev
    b = Batch(6, [(2, 600)], 64, 128, 601, 0, sink=False)
    ramp = ref.bf16(np.linspace(-1, 1, 601)[:, None] * np.ones((1, D)))
    for j in range(601):
        b.kv[int(b.table[0, j // PAGE]) * PAGE + j % PAGE] = ramp[j]
    b.q[:] = ref.bf16(np.full((2, 64, D), 8.0) * (1 + np.arange(64)[None, :, None] / 16))
    b.device(torch, dev).call()
    b.check(torch)


def test_repeatable_on_another_stream_and_in_a_graph(torch_dev):
    """The same call gives the same bits, on another stream, captured and
    replayed on new inputs, and on two streams at once with a workspace each."""
    torch, dev = torch_dev
    b = Batch(8, [(1, 3000), (1, 100), (2, 777)], 64, 512, 2000, 4).device(torch, dev)
    b.call()
    b.check(torch)
    want = [b.d["out"].clone(), b.kw["lse_out"].clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x in (b.d["out"], b.kw["lse_out"]):
            x.zero_()
        b.call()
    s.synchronize()
    assert torch.equal(want[0], b.d["out"]) and torch.equal(want[1], b.kw["lse_out"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call()
    c = Batch(9, [(1, 3000), (1, 100), (2, 777)], 64, 512, 2000, 4).device(torch, dev)
    for key in b.d:
        if key != "out":
            b.d[key].copy_(c.d[key])
    for key in ("seq", "cells", "cell_pool", "sink_logit"):
        b.kw[key].copy_(c.kw[key])
    g.replay()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(b.d["out"], c.d["out"]) and torch.equal(b.kw["lse_out"], c.kw["lse_out"])
    c.check(torch)
    want = c.d["out"].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.call()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(b.d["out"], want) and torch.equal(c.d["out"], want)


def test_out_of_range_ids_are_skipped_and_flagged(torch_dev):
    """Bad pages, cells, rows of the table and positions are no keys, and set
    FM_DEVERR_PAGE_RANGE; the rest of the call is as without them."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    b = Batch(11, [(2, 300), (2, 400)], 64, 64, 200, 4).device(torch, dev)
    b.call()
    b.check(torch)
    table, cells, seq, pos = b.table.copy(), b.cells.copy(), list(b.seq), list(b.pos)

    def again(**new):
        for name, value in new.items():
            (b.d if name in b.d else b.kw)[name].copy_(torch.from_numpy(np.asarray(value)).to(dev))
        b.call()
        torch.cuda.synchronize()
        assert fm.fm_device_status(reset=True) == fm.FM_DEVERR_PAGE_RANGE
        b.rows = [b.token_rows(t) for t in range(b.T)]
        b.check(torch)
    # a page at P and one far past it, in the windows
    b.table[0, 4], b.table[1, 5] = -1, -1
    bad = b.table.copy()
    bad[0, 4], bad[1, 5] = b.P, 2 ** 31 - 1
    again(page_table=bad)
    # cells at the pool's end and far past it
    b.cells[0, 3], b.cells[3, 0] = -1, -1
    bad = b.cells.copy()
    bad[0, 3], bad[3, 0] = b.Pc * PAGE, 2 ** 31 - 1
    (b.d["page_table"]).copy_(torch.from_numpy(b.table).to(dev))
    again(cells=bad)
    b.kw["cells"].copy_(torch.from_numpy(b.cells).to(dev))
    # a row at B
    b.seq = [seq[0], -1, seq[2], seq[3]]
    again(seq=np.array([seq[0], b.B, seq[2], seq[3]], np.int32))
    b.kw["seq"].copy_(torch.from_numpy(np.array(b.seq, np.int32)).to(dev))
    # a position past the table: the tokens past it are no keys
    far = b.R * PAGE + 40
    b.pos = [pos[0], pos[1], pos[2], far]
    b.rows = None
    b.d["pos"].copy_(torch.from_numpy(np.array(b.pos, np.int64)).to(dev))
    b.token_rows_plain = b.token_rows
    slots = [j for j in ref.visible(far, b.window, b.n_sink, b.R * PAGE)]
    b.kv[[int(b.table[1, j // PAGE]) * PAGE + j % PAGE for j in slots if b.table[1, j // PAGE] >= 0]] = ref.bf16(np.ones((1, D)))
    b.d["kv_pool"].copy_(torch.from_numpy(b.kv.view(np.int16).reshape(-1, PAGE, D)).to(dev))
    b.call()
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == fm.FM_DEVERR_PAGE_RANGE
    b.token_rows = lambda t: ([int(b.table[1, j // PAGE]) * PAGE + j % PAGE for j in slots if b.table[1, j // PAGE] >= 0]
                              if t == 3 else b.token_rows_plain(t))
    b.rows = [b.token_rows(t) for t in range(b.T)]
    b.check(torch)


def test_pools_past_32_bit_offsets(torch_dev):
    """Pages whose byte and element offsets pass 2^32."""
    torch, dev = torch_dev
    P = (1 << 32) // (PAGE * D) + 64  # elements past 2^32: 8.6 GB
    b = Batch(12, [(2, 200)], 64, 128, 150, 4)
    b.device(torch, dev)
    big = torch.empty((P, PAGE, D), dtype=torch.int16, device=dev)
    shift = P - max(b.P, b.Pc)
    big[shift:shift + b.P] = b.d["kv_pool"]
    table = torch.from_numpy(np.where(b.table >= 0, b.table + shift, -1).astype(np.int32)).to(dev)
    b.d.update(kv_pool=big, page_table=table)
    b.call()
    b.check(torch)
    big[shift:shift + b.Pc] = b.kw["cell_pool"]
    b.device(torch, dev)
    b.kw.update(cell_pool=big, cells=torch.from_numpy(np.where(b.cells >= 0, b.cells + shift * PAGE, -1).astype(np.int32)).to(dev))
    b.call()
    b.check(torch)


def test_huge_window_and_position(torch_dev):
    """A window of 2^62 tokens at a far position walks the table's pages only."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    b = Batch(13, [(1, 300)], 64, 0, 1 << 62, 2 ** 31 - 1).device(torch, dev)
    b.call()
    b.check(torch)
    assert fm.fm_device_status(reset=True) == 0


def test_no_sequences_and_nothing_to_do(torch_dev):
    """No pages, no cells, no table: every row is empty; T = 0 does nothing."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    q = torch.ones((3, 4, D), dtype=torch.bfloat16, device=dev)
    pool = torch.empty((0, PAGE, D), dtype=torch.bfloat16, device=dev)
    table = torch.empty((3, 0), dtype=torch.int32, device=dev)
    pos = torch.tensor([-1, -5, -1], device=dev)
    out, lse = torch.ones_like(q), torch.zeros((3, 4), device=dev)
    ws = torch.empty(fm.fm_csa_attn_workspace(3, 4), dtype=torch.uint8, device=dev)
    fm.fm_csa_attn(q, pool, table, pos, out, 128, lse_out=lse, sink_logit=torch.zeros(4, device=dev), workspace=ws)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert fm.fm_device_status(reset=True) == 0
    fm.fm_csa_attn(q[:0], pool, table, pos[:0], out[:0], 128)


def test_wider_pool_views_and_default_rows(torch_dev):
    """Without seq, token t reads row t of the table; layers interleaved in one
    pool are reached by the page stride."""
    torch, dev = torch_dev
    b = Batch(14, [(1, 90), (1, 130), (1, 3)], 64, 32, 100, 4, gap=5).device(torch, dev)
    b.kw["seq"] = None
    b.call()
    b.check(torch)


def test_many_short_items(torch_dev):
    """Far more tokens than SMs, each with none to three tiles of keys, so that a
    CTA goes from item to item all the time: right, and the same bits each time."""
    torch, dev = torch_dev
    seqs = [(int(n), int(n) - 1 + 7 * i) for i, n in enumerate(np.random.default_rng(3).integers(1, 60, 60))]
    b = Batch(21, seqs, 3, 40, 70, 2, Pc=4, pads=5, holes=True).device(torch, dev)
    b.call()
    b.check(torch)
    want = b.d["out"].clone()
    for _ in range(20):
        b.d["out"].zero_()
        b.call()
        torch.cuda.synchronize()
        assert torch.equal(want, b.d["out"])


@pytest.mark.parametrize("tokens", [1, 9, 19, 38, 60, 77])
def test_every_way_of_splitting(torch_dev, tokens):
    """Clusters of eight, four and two CTAs, partial results through memory, and no
    split: each with tokens whose keys leave some of the splits empty."""
    torch, dev = torch_dev
    seqs = [(1, 5000 if i % 5 == 0 else 31 * i) for i in range(tokens)]
    for window in (300, 5001):
        b = Batch(30 + tokens, seqs, 5, 16, window, 4, pads=1).device(torch, dev)
        b.call()
        b.check(torch, tokens=list(range(0, b.T, max(1, b.T // 9))) + [b.T - 1])


def test_partial_results_in_a_graph(torch_dev):
    """The split through memory (two kernels): captured, replayed on new inputs,
    and the same bits as the eager call."""
    torch, dev = torch_dev
    b = Batch(40, [(1, 7000), (1, 6500)], 64, 0, 6800, 4).device(torch, dev)
    b.call()
    b.check(torch)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call()
    c = Batch(41, [(1, 7000), (1, 6500)], 64, 0, 6800, 4).device(torch, dev)
    for key in ("q", "kv_pool", "page_table"):
        b.d[key].copy_(c.d[key])
    b.kw["sink_logit"].copy_(c.kw["sink_logit"])
    c.call()
    for _ in range(3):
        b.d["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.d["out"], c.d["out"]) and torch.equal(b.kw["lse_out"], c.kw["lse_out"])
    c.check(torch)


def test_extreme_positions_windows_and_sinks(torch_dev):
    """Nothing overflows at the ends of the types, and only tokens that a call can
    see past the table are flagged."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    b = Batch(50, [(1, 300)], 8, 20, 0, 0, sink=False).device(torch, dev)
    for pos, window, n_sink, flag in ((2 ** 63 - 1, 0, 0, 0), (2 ** 63 - 1, 0, 3, 0), (2 ** 63 - 1, 1, 0, 1),
                                      (2 ** 63 - 1, 2 ** 63 - 1, 0, 1), (b.R * PAGE - 1, 5, 2 ** 31 - 1, 0),
                                      (b.R * PAGE, 0, 2 ** 31 - 1, 1), (b.R * PAGE + 9, 3, 4, 1)):
        slots = [j for j in range(b.R * PAGE) if j <= pos and (j < n_sink or j > pos - window)]
        rows = [int(b.table[0, j // PAGE]) * PAGE + j % PAGE for j in slots]
        b.kv[rows] = ref.bf16(np.random.default_rng(1).standard_normal((len(rows), D)))
        b.d["kv_pool"].copy_(torch.from_numpy(b.kv.view(np.int16).reshape(-1, PAGE, D)).to(dev))
        b.d["pos"].fill_(pos)
        b.kw.update(window=window, n_sink=n_sink)
        b.rows = [rows]
        b.call()
        torch.cuda.synchronize()
        assert fm.fm_device_status(reset=True) == (fm.FM_DEVERR_PAGE_RANGE if flag else 0), (pos, window, n_sink)
        b.check(torch)
    # a tree whose base is past everything sees its window's tokens of the table, and flags the others
    t = Batch(51, [(4, 100)], 8, 0, 40, 0, tree=True).device(torch, dev)
    t.kw["tree_base"].fill_(2 ** 63 - 1)
    t.call()
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == fm.FM_DEVERR_PAGE_RANGE


def test_not_finite_keys_that_are_seen(torch_dev):
    """An infinite element of a visible cell makes the heads that weigh it
    infinite or NaN, and no other token's rows."""
    torch, dev = torch_dev
    b = Batch(60, [(6, 300)], 64, 32, 64, 4).device(torch, dev)
    b.call()
    b.check(torch)
    clean = b.d["out"].clone()
    row = int(b.cells[2][b.cells[2] >= 0][0])
    users = [t for t in range(b.T) if row in b.cells[t]]
    b.kw["cell_pool"].view(-1, D)[row, 5] = 0x7F80  # +inf
    b.call()
    torch.cuda.synchronize()
    out = b.d["out"]
    for t in range(b.T):
        if t in users:
            assert not torch.isfinite(out[t].view(torch.bfloat16)).all()
        else:
            assert torch.equal(out[t], clean[t])


def test_the_layer_from_selection_to_output(torch_dev):
    """As a decode step runs it: the indexer's top-k picks cells (reserve cells), the
    norm and rotation make the queries and write the token's own cell, and the
    attention reads both -- one stream, no synchronisation in between."""
    torch, dev = torch_dev
    import gen
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(70)
    t = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a if dt is None else a.view(dt))).to(dev)
    pc = gen.PagedCfg("layer", requests=5, layers=1, n_pages=30, R=9, seed=gen.BASE_SEED + 300)
    logical, phys, owner = gen.paged_tables(pc)
    pq, pw = gen.paged_qw(pc)
    k8, scale = gen.paged_pool_host(pc, owner)
    Q, H, window, n_sink = pc.Q, 64, 128, 4
    cells = torch.empty((Q, 128), dtype=torch.int32, device=dev)
    ws = torch.empty(fm.fm_native_topk_paged_workspace(Q, pc.R), dtype=torch.uint8, device=dev)
    pos = 200 + 97 * np.arange(Q)
    R = int(pos.max()) // PAGE + 1
    table = rng.permutation(Q * R).reshape(Q, R).astype(np.int32)
    kv = ref.bf16(rng.standard_normal((Q * R, PAGE, D)))
    pool = ref.bf16(rng.standard_normal((k8.shape[0], PAGE, D)))
    q, k = ref.bf16(rng.standard_normal((Q, H, D))), ref.bf16(rng.standard_normal((Q, 1, D)))
    qg, kg = ref.bf16(1 + 0.1 * rng.standard_normal(D)), ref.bf16(1 + 0.1 * rng.standard_normal(D))
    own = table[np.arange(Q), pos // PAGE] * PAGE + pos % PAGE
    kv_d, q_out = t(kv, np.int16), torch.empty((Q, H, D), dtype=torch.int16, device=dev)
    out, lse = torch.empty_like(q_out), torch.empty((Q, H), device=dev)
    aws = torch.empty(fm.fm_csa_attn_workspace(Q, H), dtype=torch.uint8, device=dev)
    args = [t(pq, np.int16), t(pw), t(k8), t(scale), t(phys), t(logical)]
    q_d, k_d, qg_d, kg_d, pos_d, own_d, tab_d, pool_d = (t(q, np.int16), t(k, np.int16), t(qg, np.int16),
                                                          t(kg, np.int16), t(pos), t(own.astype(np.int32)), t(table),
                                                          t(pool, np.int16))
    sink = torch.zeros(H, device=dev)

    def step():
        fm.fm_native_topk_paged_ex(*args, 128, cells, id_mode=1, workspace=ws)
        fm.fm_qk_norm_rope(pos_d, q=q_d, q_gain=qg_d, q_out=q_out, k=k_d, k_gain=kg_d, k_pool=kv_d, k_cell=own_d)
        fm.fm_csa_attn(q_out, kv_d, tab_d, pos_d, out, window=window, n_sink=n_sink, cell_pool=pool_d, cells=cells,
                       sink_logit=sink, lse_out=lse, workspace=aws)
    step()
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    eager = out.clone()
    # the attention's own inputs are the bits that the steps before wrote
    got_q = ref.f64(q_out.cpu().numpy().view(np.uint16))
    want_q, tol_q = ref.norm_rope(ref.f64(q), ref.f64(qg), pos, 64, 1e-6)
    assert (np.abs(got_q - want_q) <= tol_q).all()
    kv_now = kv_d.cpu().numpy().view(np.uint16).reshape(-1, D)
    want_k, tol_k = ref.norm_rope(ref.f64(k), ref.f64(kg), pos, 64, 1e-6)
    assert (np.abs(ref.f64(kv_now[own]) - want_k[:, 0]) <= tol_k[:, 0]).all()
    chosen, got = cells.cpu().numpy(), ref.f64(out.cpu().numpy().view(np.uint16))
    assert (chosen >= 0).sum(1).min() == 128
    for i in range(Q):
        slots = ref.visible(int(pos[i]), window, n_sink, int(pos[i]) + 1)
        rows = [int(table[i, j // PAGE]) * PAGE + j % PAGE for j in slots]
        keys = np.concatenate([kv_now[rows], pool.reshape(-1, D)[chosen[i]]])
        w, w_lse, tol, ltol = ref.attend(got_q[i], ref.f64(keys), np.zeros(H), D ** -0.5)
        assert (np.abs(got[i] - w) <= tol).all() and (np.abs(lse[i].cpu().numpy() - w_lse) <= ltol).all()
    # the whole step captured and replayed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and fm.fm_device_status(reset=True) == 0


@pytest.mark.parametrize("H", [2, 15, 17, 31, 32, 33, 48, 49, 63, 80, 97])
@pytest.mark.parametrize("seqs,window", [([(1, 2600)], 2601),    # through memory
                                         ([(30, 300)], 150),     # by clusters
                                         ([(200, 230)], 100)])   # several items to a CTA
def test_head_counts(torch_dev, H, seqs, window):
    """Head blocks that are not full, with a maximum that moves: nothing of the
    heads that are not there gets into the others."""
    torch, dev = torch_dev
    b = Batch(500 + H + window, seqs, H, 40, window, 2, magnitude=6.0).device(torch, dev)
    b.call()
    b.check(torch)


def test_numbers_past_their_type_are_refused(torch_dev):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    q, pos = torch.zeros((2, 4, D), dtype=torch.bfloat16, device=dev), torch.zeros(2, dtype=torch.int64, device=dev)
    with pytest.raises(ValueError):
        fm.fm_qk_norm_rope(pos, q=q, q_out=q.clone(), rope_dim=1 << 40)
    args = dict(q=q, kv_pool=torch.zeros((3, PAGE, D), dtype=torch.bfloat16, device=dev), pos=pos, out=q.clone(),
                page_table=torch.zeros((2, 2), dtype=torch.int32, device=dev))
    for bad in (dict(window=1 << 70), dict(window=8, n_sink=1 << 40)):
        with pytest.raises(ValueError):
            fm.fm_csa_attn(**args, **bad)


@pytest.mark.parametrize("seqs,H,window", [([(1, 2600)], 64, 2601), ([(30, 300)], 80, 150), ([(200, 230)], 64, 100)])
def test_output_over_the_queries(torch_dev, seqs, H, window):
    """out may be q: through memory, by clusters, several items to a CTA."""
    torch, dev = torch_dev
    b = Batch(900 + H + window, seqs, H, 40, window, 2).device(torch, dev)
    b.d["out"] = b.d["q"]
    b.call()
    b.check(torch)
