"""fm_kv_attn_fp8 against the fp64 formula: lengths from nothing to many pages, groups, windows, sinks, drafted
tokens, garbage in every cell that is no key, strides, padded batches, graphs."""
import numpy as np
import pytest

import attn_ref as ref
import grouped_ref as gr

pytestmark = pytest.mark.gpu
FOREVER = 1 << 62


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def up(torch, dev, a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def make(rng, lens, starts, H, K, d, layers=1, spread=0.3, drop=(), free=0, quick=False):
    """A cache with NaN codes and NaN scales in every cell and block that holds no token, and its fp64 values."""
    B = len(lens)
    ends = [max(s + n, 0) for n, s in zip(lens, starts)]
    R = max([(e + 63) // 64 for e in ends] + [1]) + free
    P = B * R + 2
    table = rng.permutation(P)[:B * R].reshape(B, R).astype(np.int32)
    codes = np.full((2, P, layers, K, 64, d), 0x7F, np.uint8)
    scales = np.full((2, P, layers, K, 4), np.nan, np.float32)
    mid = layers // 2
    k, v, size, scale_of, held = [], [], [], [], []
    for b in range(B):
        m = ends[b]
        if quick:  # the codes of 4096 normal values, over and over
            some = gr.e4m3_codes(np.clip(100 * rng.standard_normal(4096), -448, 448))
            c = some[rng.integers(0, 4096, (2, R * 64, K, d), dtype=np.uint16)]
        else:
            c = rng.integers(0, 256, (2, R * 64, K, d)).astype(np.uint8)
            c[(c & 127) == 127] = 0
            normal = gr.e4m3_codes(np.clip(100 * rng.standard_normal((2, R * 64, K, d)), -448, 448))
            c = np.where(rng.random((2, R * 64, K, 1)) < 0.1, c, normal)
        s = (np.exp(spread * rng.standard_normal((2, R * 4, K))) * 0.01).astype(np.float32)
        ok = np.ones(m, bool)
        for page in range(R):
            if (b, page) in drop:
                ok[page * 64:(page + 1) * 64] = False
                table[b, page] = -1
                continue
            at = table[b, page]
            rows = min(64, max(0, m - page * 64))
            codes[:, at, mid, :, :rows] = c[:, page * 64:page * 64 + rows].transpose(0, 2, 1, 3)
            for blk in range(4):
                if page * 64 + blk * 16 < m:
                    scales[:, at, mid, :, blk] = s[:, page * 4 + blk]
        j = np.arange(m)
        x = gr.VALUES[c[:, :m]] * s.astype(np.float64)[:, j // 16][..., None]
        k.append(x[0])
        v.append(x[1])
        size.append(np.abs(gr.VALUES[c[1, :m]]))
        scale_of.append(s[1].astype(np.float64)[j // 16][..., None])
        held.append(ok)
    return table, codes, scales, k, v, size, scale_of, held


def check(torch, dev, rng, lens, starts, H, K, d, window=None, sink=False, layers=1, pad=0, offsets=True, scale=None, **kw):
    import sparse_attention_kv_c4_gb300 as fm
    flags = kw.pop("flags", 0)
    q_size = kw.pop("q_size", 1.0)
    table, codes, scales, k, v, size, scale_of, held = make(rng, lens, starts, H, K, d, layers, **kw)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + pad
    fused = ref.bf16(q_size * rng.standard_normal((T, H * d + 16)))
    q = up(torch, dev, fused.view(np.int16))[:, :H * d].view(T, H, d)
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    mid = layers // 2
    sinks = rng.standard_normal(H).astype(np.float32) if sink else None
    out = torch.full((T, H, d), 77, dtype=torch.int16, device=dev)
    lse = torch.full((T, H), 77.0, device=dev)
    ws = torch.empty(max(fm.fm_kv_attn_fp8_workspace(T, H, K, d), 1), dtype=torch.uint8, device=dev)
    ws.fill_(0xFF)
    fm.fm_kv_attn_fp8(q, cd[0][:, mid], cd[1][:, mid], sd[0][:, mid], sd[1][:, mid], up(torch, dev, table),
                      up(torch, dev, np.array(starts, np.int64)), out, cu_tokens=up(torch, dev, cu) if offsets else None, window=window,
                      sink_logit=None if sinks is None else up(torch, dev, sinks), scale=scale, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == flags
    got, got_lse = out.cpu().numpy().view(np.uint16), lse.cpu().numpy().astype(np.float64)
    assert (got[cu[-1]:] == 77).all() and (got_lse[cu[-1]:] == 77).all()
    qf = ref.f64(fused[:, :H * d]).reshape(T, H, d)
    for b, (n, s) in enumerate(zip(lens, starts)):
        rows = slice(cu[b], cu[b + 1])
        want, want_lse, tol, ltol = gr.attend(qf[rows], k[b], v[b], s, FOREVER if window is None else window, sinks,
                                              d ** -0.5 if scale is None else scale, held[b], gr.HALF_FP16, (size[b], scale_of[b]))
        g, gl = ref.f64(got[rows]), got_lse[rows]
        empty = np.isneginf(want_lse)
        assert (np.isneginf(gl) == empty).all() and (g[empty] == 0).all()
        assert (np.abs(gl[~empty] - want_lse[~empty]) <= ltol[~empty]).all(), b
        assert (np.abs(g - want) <= tol).all(), (b, np.abs(g - want).max())


@pytest.mark.parametrize("lens,starts,H,K,d,window,sink", [
    ([1], [0], 1, 1, 16, None, False), ([1], [36], 32, 8, 128, None, False), ([1] * 5, [0, 15, 16, 63, 64], 8, 8, 64, None, True),
    ([1] * 7, [127, 300, 1, 700, 64, 65, 2000], 20, 4, 96, None, True), ([1] * 3, [900, 77, 4000], 64, 8, 128, 129, False),
    ([1] * 3, [900, 77, 4000], 5, 1, 128, 1, True), ([1, 1], [50, 60], 4, 2, 32, 0, True), ([5] * 4, [0, 60, 123, 1000], 40, 8, 64, None, True),
    ([3, 0, 8, 1], [10, 4, 300, 129], 6, 2, 112, 70, False), ([17, 2], [40, 500], 16, 1, 48, None, False), ([2, 130], [1, 5], 12, 4, 128, 65, True),
    ([1], [9000], 128, 1, 128, None, False), ([1, 4], [33000, 900], 8, 2, 80, None, True), ([7], [20], 128, 1, 64, 9, True)])
def test_matches_formula(torch_dev, lens, starts, H, K, d, window, sink):
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(H + d + len(lens)), lens, starts, H, K, d, window, sink)


def test_padded_batch_layers_between_and_no_offsets(torch_dev):
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(1), [1, 3, 1], [200, 100, 30], 8, 2, 64, layers=3, pad=5)
    check(torch, dev, np.random.default_rng(2), [1] * 9, [31 * b for b in range(9)], 8, 2, 128, layers=2, offsets=False)


def test_pages_not_held_and_out_of_range(torch_dev):
    torch, dev = torch_dev
    rng = np.random.default_rng(3)
    check(torch, dev, rng, [1, 2, 1, 1], [300, 200, 70, 64], 8, 2, 64, drop={(0, 1), (0, 3), (1, 0), (2, 0), (2, 1), (3, 1)}, free=1)
    check(torch, dev, rng, [2, 1], [-2, -1], 4, 2, 64)


def test_tables_that_are_too_short_or_name_no_page_are_flagged(torch_dev):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(4)
    table, codes, scales, k, v, size, scale_of, held = make(rng, [1, 1], [150, 20], 4, 2, 64)
    table[0, 1] = codes.shape[1] + 7
    held[0][64:128] = False
    q = ref.bf16(rng.standard_normal((2, 4, 64)))
    out, ws = torch.zeros((2, 4, 64), dtype=torch.int16, device=dev), torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(2, 4, 2, 64)), dtype=torch.uint8, device=dev)
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    for start in ([150, 20], [5 * 64, 20], [1 << 61, 20]):  # the first sequence's last tokens lie past the table
        st = torch.tensor(start, device=dev)
        fm.fm_kv_attn_fp8(up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table), st, out, workspace=ws)
        assert fm.fm_device_status(reset=True) == 1
    got = ref.f64(out.cpu().numpy().view(np.uint16))
    want, _, tol, _ = gr.attend(ref.f64(q)[1:], k[1], v[1], 20, FOREVER, None, 0.125, held[1], gr.HALF_FP16, (size[1], scale_of[1]))
    assert (np.abs(got[1:] - want) <= tol).all()


def test_scales_of_every_size(torch_dev):
    """Values whose blocks' scales differ by e^30, scores of hundreds, queries near the ends of bf16."""
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(5), [1, 3], [500, 90], 8, 2, 64, spread=8.0, scale=1e-6)
    check(torch, dev, np.random.default_rng(6), [1, 3], [500, 90], 8, 2, 64, scale=60.0)
    check(torch, dev, np.random.default_rng(7), [1, 3], [500, 90], 8, 2, 64, q_size=1e30, scale=1e-30)
    check(torch, dev, np.random.default_rng(8), [1, 3], [500, 90], 8, 2, 64, q_size=1e-30, scale=1e30)


def test_a_drafted_token_does_not_see_what_a_later_one_holds(torch_dev):
    """The last draft's cell and scale are NaN: the earlier drafts' rows are as without it, its own row is NaN."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(11)
    for start in (64, 40, 60, 15):  # the drafts within a block, over a block's and a page's border
        table, codes, scales, k, v, size, scale_of, held = make(rng, [4], [start], 8, 2, 64)
        last = start + 3
        codes[1, table[0, last // 64], 0, 1, last % 64, 5] = 0x7F
        q = ref.bf16(rng.standard_normal((4, 8, 64)))
        out, ws = torch.zeros((4, 8, 64), dtype=torch.int16, device=dev), torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(4, 8, 2, 64)), dtype=torch.uint8, device=dev)
        cd, sd = up(torch, dev, codes), up(torch, dev, scales)
        fm.fm_kv_attn_fp8(up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table),
                          torch.tensor([start], device=dev), out, cu_tokens=torch.tensor([0, 4], dtype=torch.int32, device=dev), workspace=ws)
        got = ref.f64(out.cpu().numpy().view(np.uint16))
        assert np.isnan(got[3, 4:, 5]).all() and np.isnan(got).sum() == 4
        want, _, tol, _ = gr.attend(ref.f64(q)[:3], k[0], v[0], start, FOREVER, None, 0.125, held[0], gr.HALF_FP16, (size[0], scale_of[0]))
        assert (np.abs(got[:3] - want) <= tol).all()


def test_long_caches_see_every_key(torch_dev):
    """One long sequence beside short ones: a single key of another value among equal ones is found at every
    place where the work may be split."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    d, K, H, m = 64, 2, 8, 40000
    R = (m + 63) // 64
    codes = torch.zeros((2, R + 1, K, 64, d), dtype=torch.uint8, device=dev)
    scales = torch.full((2, R + 1, K, 4), 2.0, device=dev)
    table = torch.stack([torch.randperm(R), torch.cat([torch.tensor([R]), torch.full((R - 1,), -1)])]).int().to(dev)
    start = torch.tensor([m - 1, 10], device=dev)
    q = torch.randn((2, H, d), device=dev).bfloat16()
    out, lse = torch.empty((2, H, d), dtype=torch.bfloat16, device=dev), torch.empty((2, H), device=dev)
    ws = torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(2, H, K, d)), dtype=torch.uint8, device=dev)
    places = sorted({0, 1, 15, 16, 63, 64, 65, m - 1, m - 2} | {int(x) for x in np.random.default_rng(0).integers(0, m, 60)})
    for j in places:
        page, row = int(table[0, j // 64]), j % 64
        codes[1, page, :, row] = 0x7E  # 448
        fm.fm_kv_attn_fp8(q, codes[0], codes[1], scales[0], scales[1], table, start, out, lse_out=lse, workspace=ws)
        codes[1, page, :, row] = 0
        want = 448 * 2.0 / m  # weights are equal: keys are zero
        got = out[0].double().cpu().numpy()
        assert (np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9)).all(), j
        assert (out[1] == 0).all().item()
    assert np.abs(lse.cpu().numpy()[0] - np.log(m)).max() <= 2.0 ** -19 * 11 + m * 2.0 ** -24


@pytest.mark.parametrize("H,K,d,lens,starts,window", [
    (8, 8, 64, [1, 1, 1], [24000, 35, 21003], None), (8, 8, 128, [1, 2], [18001, 9000], None), (10, 2, 96, [2, 1, 5], [24000, 30000, 9], 20001)])
def test_many_pages_to_each_sm(torch_dev, H, K, d, lens, starts, window):
    """Runs that go round their stages many times, several heads and sequences to a run; twenty calls give
    the same bits."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(H)
    table, codes, scales, k, v, size, scale_of, held = make(rng, lens, starts, H, K, d, quick=True)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q = ref.bf16(rng.standard_normal((T, H, d)))
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    args = (up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table), torch.tensor(starts, device=dev))
    out, lse = torch.zeros((T, H, d), dtype=torch.int16, device=dev), torch.zeros((T, H), device=dev)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(T, H, K, d), dtype=torch.uint8, device=dev)
    first = None
    for _ in range(20):
        out.zero_()
        fm.fm_kv_attn_fp8(*args, out, cu_tokens=up(torch, dev, cu), window=window, lse_out=lse, workspace=ws)
        torch.cuda.synchronize()
        first = out.clone() if first is None else first
        assert (out == first).all().item()
    assert fm.fm_device_status(reset=True) == 0
    got, got_lse = ref.f64(out.cpu().numpy().view(np.uint16)), lse.double().cpu().numpy()
    for b in range(len(lens)):
        rows = slice(cu[b], cu[b + 1])
        want, want_lse, tol, ltol = gr.attend(ref.f64(q)[rows], k[b], v[b], starts[b], FOREVER if window is None else window, None, d ** -0.5,
                                              held[b], gr.HALF_FP16, (size[b], scale_of[b]))
        assert (np.abs(got_lse[rows] - want_lse) <= ltol).all() and (np.abs(got[rows] - want) <= tol).all(), b


@pytest.mark.parametrize("T,H,K,d", [(1, 24, 1, 64), (3, 8, 1, 48), (1, 17, 1, 64), (1, 24, 1, 128), (2, 9, 1, 128), (1, 128, 1, 64), (5, 5, 1, 64)])
def test_the_workspace_holds_what_is_written(torch_dev, T, H, K, d):
    """Rows that do not fill their eights, split over every SM: nothing is written behind the workspace's end."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(T + H)
    starts = [9000] * T
    table, codes, scales, k, v, size, scale_of, held = make(rng, [1] * T, starts, H, K, d, quick=True)
    need = fm.fm_kv_attn_fp8_workspace(T, H, K, d)
    ws = torch.full((need + (1 << 24),), 0xA5, dtype=torch.uint8, device=dev)
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    q = ref.bf16(rng.standard_normal((T, H, d)))
    out = torch.zeros((T, H, d), dtype=torch.int16, device=dev)
    fm.fm_kv_attn_fp8(up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table),
                      torch.tensor(starts, device=dev), out, workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0xA5).all().item() and fm.fm_device_status(reset=True) == 0
    got = ref.f64(out.cpu().numpy().view(np.uint16))
    want, _, tol, _ = gr.attend(ref.f64(q)[:1, :4], k[0], v[0], 9000, FOREVER, None, d ** -0.5, held[0], gr.HALF_FP16, (size[0], scale_of[0]))
    assert (np.abs(got[:1, :4] - want) <= tol).all()


def test_two_calls_at_once_graph_and_same_results(torch_dev):
    """The result is the same bits eager, replayed on another stream, and beside another call with a workspace
    of its own; out may be q."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(12)
    cases = []
    for starts, H, K, d in (([5000, 100, 7000], 16, 4, 128), ([300, 9000], 8, 8, 64)):
        table, codes, scales = make(rng, [1] * len(starts), starts, H, K, d)[:3]
        T = len(starts)
        cd, sd = up(torch, dev, codes), up(torch, dev, scales)
        q = torch.randn((T, H, d), device=dev).bfloat16()
        args = (cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table), torch.tensor(starts, device=dev))
        ws = torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(T, H, K, d)), dtype=torch.uint8, device=dev)
        want = torch.empty_like(q)
        fm.fm_kv_attn_fp8(q, *args, want, workspace=ws)
        cases.append((q, args, ws, want))
    streams = [torch.cuda.Stream(dev) for _ in cases]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for (q, args, ws, want), s in zip(cases, streams):
        g, out = torch.cuda.CUDAGraph(), q.clone()
        with torch.cuda.graph(g, stream=s):
            fm.fm_kv_attn_fp8(out, *args, out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for _ in range(5):
        for (q, *_), out in zip(cases, outs):
            out.copy_(q)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, want), out in zip(cases, outs):
            assert (out.view(torch.int16) == want.view(torch.int16)).all()
    assert fm.fm_device_status(reset=True) == 0


@pytest.mark.parametrize("B,K,G,n,d", [(133, 8, 1, 1, 64), (133, 8, 2, 1, 128), (70, 16, 16, 1, 64), (70, 16, 2, 8, 128),
                                       (36, 16, 6, 4, 128), (36, 16, 8, 4, 64)])
@pytest.mark.parametrize("above,place", [(12.0, 0), (17.5, 0), (17.5, 2000), (17.5, 4080), (60.0, 0), (60.0, 2000)])
def test_keys_under_one_that_takes_nearly_all_of_the_weight(torch_dev, B, K, G, n, d, above, place):
    """A key whose score is `above` nats over the others' and whose value is zero, by itself and in a block of 64 times the
    scale: the output is that of the others.  Requests share their 64 pages, so that each warp has all of a request's.

    Values are positive, so that bounds are relative: a weight times scale is off by 2^-11 of itself, or by 2^-22 of the largest
    of its page but by no more than itself; scores and sums as in grouped_ref.attend; half a step of bf16."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    m, H, T = 4096, K * G, B * n
    g = torch.Generator(device=dev).manual_seed(B + d)
    k = (32 * torch.randn((64, K, 64, d), generator=g, device=dev) * 0.5).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    k[..., 0] = 0
    k[place // 64, :, place % 64] = 0
    k[place // 64, :, place % 64, 0] = 0x7E  # 448
    v = torch.randint(0x60, 0x70, (64, K, 64, d), generator=g, device=dev, dtype=torch.uint8)  # 32 .. 60
    v[place // 64, :, place % 64] = 0
    table = torch.randperm(64, generator=g, device=dev).int()
    inverse = torch.empty_like(table)
    inverse[table.long()] = torch.arange(64, device=dev, dtype=torch.int32)
    q = torch.randn((T, H, d), generator=g, device=dev)
    q[..., 0] = above * d ** 0.5 / (448 / 32)
    q = q.bfloat16()
    out, lse = torch.empty_like(q), torch.empty((T, H), device=dev)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(T, H, K, d), dtype=torch.uint8, device=dev)
    for times in (1.0, 64.0):
        ks, vs = torch.full((64, K, 4), 2.0 ** -5, device=dev), torch.full((64, K, 4), 2.0 ** -6, device=dev)
        vs[place // 64, :, place % 64 // 16] *= times
        order = inverse.long()
        fm.fm_kv_attn_fp8(q, k[order], v[order], ks[order], vs[order], table.expand(B, 64).contiguous(), torch.full((B,), m - n, device=dev), out,
                          cu_tokens=torch.arange(B + 1, device=dev, dtype=torch.int32) * n, lse_out=lse, workspace=ws)
        value = lambda c, s: (c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(16, -1)[..., None]).transpose(1, 2).reshape(m, K, d)
        kf, vf = value(k, ks), value(v, vs)
        seen = torch.arange(m, device=dev) <= torch.arange(m - n, m, device=dev)[:, None]
        for h in range(K):
            rows = q.view(B, n, K, G, d)[:, :, h].transpose(1, 2).reshape(B * G, n, d).double()
            score = (rows @ kf[:, h].T * d ** -0.5).masked_fill(~seen, -float("inf"))
            size = (rows.abs() @ kf[:, h].abs().T * d ** -0.5).amax()
            w = score.softmax(-1)
            weighed = w * vs[:, h].double().repeat_interleave(16, -1).view(m)
            page = weighed.view(B * G, n, 64, 64).amax(-1, keepdim=True)
            lost = torch.minimum(2.0 ** -22 * page.expand(-1, -1, -1, 64).reshape(weighed.shape), weighed)
            codes = v[:, h].view(torch.float8_e4m3fn).double().view(m, d)
            want = w @ vf[:, h]
            rel = 2 * ((d + 8) * 2.0 ** -24 * size + 2.0 ** -22 * above) + 2.0 ** -20 + m * 2.0 ** -24
            tol = want * (2 * rel + 2.0 ** -11 + 2.0 ** -8) + lost @ codes
            got = out.view(B, n, K, G, d)[:, :, h].transpose(1, 2).reshape(B * G, n, d).double()
            assert ((got - want).abs() <= tol).all().item(), (times, h, ((got - want).norm() / want.norm()).item())
            got_lse = lse.view(B, n, K, G)[:, :, h].transpose(1, 2).reshape(B * G, n).double()
            assert ((got_lse - score.logsumexp(-1)).abs() <= 2 * rel + 2.0 ** -21 * (above + 10)).all().item()
    assert fm.fm_device_status(reset=True) == 0


def one_call(torch, dev, q, codes, scales, table, lens, starts, d, scale=None):
    """One call over arrays as make's; out and lse in fp64."""
    import sparse_attention_kv_c4_gb300 as fm
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, H, K = int(cu[-1]), q.shape[1], codes.shape[3]
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    out, lse = torch.zeros((T, H, d), dtype=torch.int16, device=dev), torch.zeros((T, H), device=dev)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(T, H, K, d), dtype=torch.uint8, device=dev)
    fm.fm_kv_attn_fp8(up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table),
                      torch.tensor(starts, device=dev), out, cu_tokens=up(torch, dev, cu), scale=scale, lse_out=lse, workspace=ws)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    return ref.f64(out.cpu().numpy().view(np.uint16)), lse.double().cpu().numpy()


@pytest.mark.parametrize("d,K,G", [(64, 2, 1), (128, 2, 2), (64, 2, 30)])
def test_values_that_shrink_from_page_to_page(torch_dev, d, K, G):
    """Scales of V from 2^90 down to 2^-100, the larger ones' values zero up to a page: the outputs are those of the first
    page that has values, whatever the references went through; and from 2^-40 up to 2^30, the later pages' zero."""
    torch, dev = torch_dev
    rng, m = np.random.default_rng(d + G), 640
    for first in (0, 3, 9):
        for turned in (False, True):
            # each request has all ten pages in one run where there are enough requests; they share them
            B = 133 * 8 // K
            table, codes, scales, k, v, size, scale_of, held = make(rng, [1], [m - 1], K * G, K, d)
            at = np.arange(m) // 64
            power = 2.0 ** (np.linspace(-40, 30, 10) if turned else np.linspace(90, -100, 10)).astype(int)
            empty = np.arange(10)[::-1 if turned else 1] < first
            scales[1][table[0]] = power[:, None, None, None]
            codes[1][table[0][empty]] = 0
            size, scale_of = size[0] * ~empty[at][:, None, None], power[at][:, None, None] * np.ones((1, K, 1))
            q = ref.bf16(rng.standard_normal((1, K * G, d))).repeat(B, 0)
            got, lse = one_call(torch, dev, q, codes, scales, table.repeat(B, 0), [1] * B, [m - 1] * B, d)
            want, want_lse, _, ltol = gr.attend(ref.f64(q)[:1], k[0], size * np.sign(v[0]) * scale_of, m - 1, FOREVER, None, d ** -0.5, held[0])
            # the page of the largest scale with values: its weights' bound for all
            top = np.flatnonzero(power * ~empty == (power * ~empty).max())[0]
            mean = size * scale_of
            s = np.einsum("hd,mhd->hm", ref.f64(q)[0], k[0].repeat(G, 1)) * d ** -0.5
            w = np.exp(s - want_lse.T)
            a = np.einsum("hm,mhd->hd", w, mean.repeat(G, 1))
            tol = a * (2.0 ** -11 + 2 * 2.0 ** -15) + 64 * 2.0 ** -22 * 448 * (w * scale_of.repeat(G, 1)[:, :, 0].T).reshape(-1, m)[:, at == top].max(1)[:, None]
            assert (np.abs(got - want) <= tol + 2.0 ** -8 * np.abs(want)).all(), (first, turned)
            assert (np.abs(lse - want_lse) <= ltol).all()


@pytest.mark.parametrize("size", [1e-36, 1e35])
def test_outputs_at_the_ends_of_the_types(torch_dev, size):
    """Scales of 2^-126 and of 2^110: outputs as small, and as large."""
    torch, dev = torch_dev
    K, G, d, rng = 2, 2, 64, np.random.default_rng(1)
    table, codes, scales, k, v, sizes, scale_of, held = make(rng, [1], [300], K * G, K, d)
    s = np.float32(2.0 ** np.floor(np.log2(size)) / 64)
    scales[1] = np.where(np.isnan(scales[1]), scales[1], s)
    scale_of = np.full_like(scale_of[0], s, dtype=np.float64)
    q = ref.bf16(rng.standard_normal((1, K * G, d)))
    got, lse = one_call(torch, dev, q, codes, scales, table, [1], [300], d)
    want, want_lse, tol, ltol = gr.attend(ref.f64(q), k[0], sizes[0] * np.sign(v[0]) * s, 300, FOREVER, None, d ** -0.5, held[0], gr.HALF_FP16,
                                          (sizes[0], scale_of))
    # grouped_ref's absolute term of 2^-120 is these outputs' size: bf16's smallest step instead
    assert (np.abs(got - want) <= tol - 2.0 ** -120 + 2.0 ** -133).all() and (np.abs(lse - want_lse) <= ltol).all()


@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 2), (128, 5)])
def test_scales_far_apart(torch_dev, d, G):
    """Values' scales of 2^-100 (a block of zeros, as the append stores it) and of 2^40: a key that a row does not see, and one
    whose weight is none in fp32, have no part in it."""
    torch, dev = torch_dev
    K, rng = 2, np.random.default_rng(d + G)
    for n, start, border in ((4, 13, 16), (4, 62, 64), (1, 127, 64)):
        table, codes, scales, k, v, size, scale_of, held = make(rng, [n], [start], K * G, K, d)
        q = ref.bf16(rng.standard_normal((n, K * G, d)))
        m = start + n
        at = np.arange(m)
        scale_of[0] = np.where(at < border, 2.0 ** -100, 2.0 ** 40)[:, None, None] * np.ones((1, K, 1))
        for b in range((m + 15) // 16):
            scales[1, table[0, b // 4], 0, :, b % 4] = 2.0 ** (-100 if 16 * b < border else 40)
        if n == 1:  # the far keys' scores lie 120 nats below
            q[..., 0] = ref.bf16(np.full(1, 120 * d ** 0.5))
            for j in range(m):
                codes[0, table[0, j // 64], 0, :, j % 64, 0] = 0 if j < border else 0xB8  # -1
                k[0][j, :, 0] = 0.0 if j < border else -1.0
            scales[0] = np.where(np.isnan(scales[0]), scales[0], 1.0)
            k[0] = gr.VALUES[codes[0][table[0, at // 64], 0, :, at % 64]]
            q[..., 1:] = ref.bf16(0.01 * rng.standard_normal((1, K * G, d - 1)))
        value = size[0] * np.sign(v[0]) * scale_of[0]
        got, lse = one_call(torch, dev, q, codes, scales, table, [n], [start], d)
        want, want_lse, tol, ltol = gr.attend(ref.f64(q), k[0], value, start, FOREVER, None, d ** -0.5, held[0], gr.HALF_FP16, (size[0], scale_of[0]))
        assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all(), (n, start, np.abs(got - want).max())
        assert (np.abs(lse - want_lse) <= ltol).all()


@pytest.mark.parametrize("which,bad", [(0, np.nan), (1, np.nan), (0, np.inf), (1, np.inf)])
def test_a_later_drafts_scale_does_not_reach_the_earlier_rows(torch_dev, which, bad):
    """A block that only the later drafts see has a scale that is no number: the rows that do not see it are as without."""
    torch, dev = torch_dev
    rng = np.random.default_rng(21)
    for start, d in ((15, 64), (62, 64), (31, 128)):
        table, codes, scales, k, v, size, scale_of, held = make(rng, [4], [start], 8, 2, d)
        border = (start // 16 + 1) * 16
        scales[which, table[0, border // 64], 0, 1, border % 64 // 16] = bad
        q = ref.bf16(rng.standard_normal((4, 8, d)))
        got, _ = one_call(torch, dev, q, codes, scales, table, [4], [start], d)
        want, _, tol, _ = gr.attend(ref.f64(q), k[0], v[0], start, FOREVER, None, d ** -0.5, held[0], gr.HALF_FP16, (size[0], scale_of[0]))
        sees = np.arange(start, start + 4) >= border
        clean = np.ones(got.shape, bool)
        clean[np.ix_(sees, range(4, 8))] = False
        assert (np.abs(got - want) <= tol)[clean].all(), (start, d)
        if np.isnan(bad):
            assert np.isnan(got[~clean]).all()


@pytest.mark.parametrize("d,G", [(64, 1), (128, 5)])
def test_scores_near_the_least_number(torch_dev, d, G):
    """Keys whose scores are -10^31 and less are keys: equal ones share the weight, the larger one has it all."""
    torch, dev = torch_dev
    K, rng = 2, np.random.default_rng(3)
    table, codes, scales, k, v, size, scale_of, held = make(rng, [1, 3], [4, 200], K * G, K, d)
    codes[0] = np.where(codes[0] == 0x7F, 0x7F, 0x40)  # 2
    scales[0] = np.where(np.isnan(scales[0]), scales[0], np.float32(1e16))
    q = ref.bf16(np.full((4, K * G, d), -1e16))
    got, lse = one_call(torch, dev, q, codes, scales, table, [1, 3], [4, 200], d)
    score = float(ref.f64(q)[0, 0, 0]) * 2 * float(np.float32(1e16)) * d * d ** -0.5
    assert (np.abs(lse / score - 1) <= 2.0 ** -18).all()
    for b, rows in ((0, range(1)), (1, range(1, 4))):
        for i, r in enumerate(rows):
            seen = v[b][:(4, 200)[b] + i + 1].repeat(G, 1)
            tol = 2.0 ** -8 * np.abs(seen.mean(0)) + (2.0 ** -11 + 2.0 ** -14) * np.abs(seen).mean(0)
            assert (np.abs(got[r] - seen.mean(0)) <= tol).all(), r
    for j in (0, 130):  # one key's score of half the size is the largest by far
        codes[0, table[1, j // 64], 0, :, j % 64] = 0x38  # 1
        got, lse = one_call(torch, dev, q, codes, scales, table, [1, 3], [4, 200], d)
        want = v[1][j].repeat(G, 0)
        assert (np.abs(got[1:] - want) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(want)).all() and (np.abs(lse[1:] / score - 0.5) <= 2.0 ** -18).all()
        codes[0, table[1, j // 64], 0, :, j % 64] = 0x40


@pytest.mark.parametrize("size", [1e6, 3e8, 1e12])
@pytest.mark.parametrize("d,G,m", [(64, 1, 40), (64, 30, 3000), (128, 2, 300), (128, 20, 3000)])
def test_scores_of_millions(torch_dev, size, d, G, m):
    """Scores whose spacing in fp32 is coarser than the weights' range, in one run and in many: out is the mean of some of the
    values, by weights that are each their own within the rounding of the score: those of the largest alone where it stands out."""
    torch, dev = torch_dev
    K, rng = 2, np.random.default_rng(int(np.log2(size)) + d + m)
    table, codes, scales, k, v, sizes, scale_of, held = make(rng, [1], [m - 1], K * G, K, d)
    scales[0] = np.where(np.isnan(scales[0]), scales[0], np.float32(size))
    at = np.arange(m)
    k[0] = gr.VALUES[codes[0][table[0, at // 64], 0, :, at % 64]] * np.float64(np.float32(size))
    q = ref.bf16(rng.standard_normal((1, K * G, d)))
    got, lse = one_call(torch, dev, q, codes, scales, table, [1], [m - 1], d)
    score = np.einsum("hd,mhd->hm", ref.f64(q)[0], k[0].repeat(G, 1)) * d ** -0.5
    bound = (d + 8) * 2.0 ** -23 * (np.einsum("hd,mhd->hm", np.abs(ref.f64(q)[0]), np.abs(k[0]).repeat(G, 1)) * d ** -0.5).max(1)
    top = score.max(1)
    assert np.isfinite(got).all() and (np.abs(lse[0] - top) <= bound + np.log(m) + 2.0 ** -21 * np.abs(top)).all()
    for h in range(K * G):
        close = score[h] >= top[h] - 2 * bound[h] - 20  # all that may be the largest, and what e^-20 leaves
        x = v[0][close, h // G]
        slack = 2.0 ** -7 * np.abs(v[0][:, h // G]).max(0) + 2.0 ** -120
        assert (got[0, h] >= x.min(0) - slack).all() and (got[0, h] <= x.max(0) + slack).all(), h


@pytest.mark.parametrize("d,G,m", [(64, 1, 40), (128, 2, 700), (64, 30, 700)])
def test_a_sink_far_over_the_scores(torch_dev, d, G, m):
    """A sink 60 to 100 nats over every score: the output is as much smaller, to the end of fp32's range, and lse is unchanged."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    K, rng = 2, np.random.default_rng(d + m)
    table, codes, scales, k, v, sizes, scale_of, held = make(rng, [1], [m - 1], K * G, K, d)
    q, H = ref.bf16(rng.standard_normal((1, K * G, d))), K * G
    cd, sd = up(torch, dev, codes), up(torch, dev, scales)
    out, lse = torch.zeros((1, H, d), dtype=torch.int16, device=dev), torch.zeros((1, H), device=dev)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(1, H, K, d), dtype=torch.uint8, device=dev)
    for over in (60.0, 88.0, 95.0, np.inf):
        sinks = np.full(H, over, np.float32)
        fm.fm_kv_attn_fp8(up(torch, dev, q.view(np.int16)), cd[0][:, 0], cd[1][:, 0], sd[0][:, 0], sd[1][:, 0], up(torch, dev, table),
                          torch.tensor([m - 1], device=dev), out, sink_logit=up(torch, dev, sinks), lse_out=lse, workspace=ws)
        want, want_lse, tol, ltol = gr.attend(ref.f64(q), k[0], v[0] * 1e3, m - 1, FOREVER, sinks, d ** -0.5, held[0], gr.HALF_FP16,
                                              (sizes[0], scale_of[0] * 1e3))
        got = ref.f64(out.cpu().numpy().view(np.uint16)) * 1e3
        # grouped_ref's absolute term of 2^-120 is these outputs' size: a step of bf16's subnormals instead; an exponential of
        # an argument of 100 is off by 2^-16
        assert (np.abs(got - want) <= tol - 2.0 ** -120 + 2.0 ** -15 * np.abs(want) + 1e3 * 2.0 ** -133).all(), over
        assert (np.abs(lse.double().cpu().numpy() - want_lse) <= ltol).all()


@pytest.mark.parametrize("d,G", [(64, 1), (128, 2), (64, 30)])
@pytest.mark.parametrize("far", [2000.0, 1e6])
def test_scores_that_rise_from_far_below_keep_their_digits(torch_dev, d, G, far):
    """The first pages' scores lie `far` below the others', in one run: the others' weights and lse are as exact as without them."""
    torch, dev = torch_dev
    K, m, B, rng = 2, 640, 532, np.random.default_rng(int(far) + d)
    table, codes, scales, k, v, size, scale_of, held = make(rng, [1], [m - 1], K * G, K, d)
    q, at = ref.bf16(rng.standard_normal((1, K * G, d))), np.arange(m)
    q[..., 0] = ref.bf16(np.full(1, far * d ** 0.5 / 4))
    codes[0][table[0], 0, :, :, 0] = 0
    codes[0][table[0][:3], 0, :, :, 0] = 0xC8  # -4, with a scale of 1 beside it
    scales[0][table[0][:3]] = 1.0
    k[0] = gr.VALUES[codes[0][table[0, at // 64], 0, :, at % 64]] * scales[0][table[0, at // 64], 0, :, at % 64 // 16].astype(np.float64)[..., None]
    got, lse = one_call(torch, dev, q.repeat(B, 0), codes, scales, table.repeat(B, 0), [1] * B, [m - 1] * B, d)
    want, want_lse, tol, ltol = gr.attend(ref.f64(q), k[0], v[0], m - 1, FOREVER, None, d ** -0.5, held[0], gr.HALF_FP16, (size[0], scale_of[0]))
    assert (np.abs(got - want) <= tol).all() and (np.abs(lse - want_lse) <= ltol).all()
