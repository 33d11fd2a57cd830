"""fm_prompt_attn against the fp64 formula: packed lengths, groups, windows, prefixes, sinks, infinities and NaN behind
the mask, strides, padded batches, graphs."""
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


def call(torch, dev, q, k, v, lens, pasts, window, sinks, scale, pad, offsets=True):
    """q, k, v bit patterns [T or Tk, heads * d + 8, ...]: slices of wider rows."""
    import sparse_attention_kv_c4_gb300 as fm
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum([n + p for n, p in zip(lens, pasts)])]).astype(np.int32)
    wide = lambda x: up(torch, dev, np.concatenate([x.reshape(len(x), x.shape[1] * x.shape[2]), np.full((len(x), 8), 0x7FC0, np.uint16)], 1).view(np.int16))[
        :, :x.shape[1] * x.shape[2]].view(x.shape)
    out = torch.full(q.shape, 77, dtype=torch.int16, device=dev)
    lse = torch.full(q.shape[:2], 77.0, device=dev)
    same = all(p == 0 for p in pasts) and pad == 0
    kw = dict(cu_q=up(torch, dev, cu), cu_k=None if same else up(torch, dev, cu_k)) if offsets else {}
    fm.fm_prompt_attn(wide(q), wide(k), wide(v), out, window=window, sink_logit=None if sinks is None else up(torch, dev, sinks), scale=scale,
                      lse_out=lse, **kw)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    return out.cpu().numpy().view(np.uint16), lse.cpu().numpy().astype(np.float64), cu, cu_k


def check(torch, dev, rng, lens, pasts, H, K, d, window=None, sink=False, scale=None, pad=0, offsets=True, rows=None, size=1.0):
    T, Tk = sum(lens) + pad, sum(lens) + sum(pasts) + 2 * pad
    q, k, v = ref.bf16(size * rng.standard_normal((T, H, d))), ref.bf16(rng.standard_normal((Tk, K, d))), ref.bf16(rng.standard_normal((Tk, K, d)))
    if pad:
        q[-pad:], k[-2 * pad:], v[-2 * pad:] = 0x7FC0, 0x7F80, 0x7FC0  # what is behind the last sequence
    sinks = rng.standard_normal(H).astype(np.float32) if sink else None
    got, lse, cu, cu_k = call(torch, dev, q, k, v, lens, pasts, window, sinks, scale, pad, offsets)
    assert (got[cu[-1]:] == 77).all() and (lse[cu[-1]:] == 77).all()
    for b, (n, past) in enumerate(zip(lens, pasts)):
        some = np.arange(n) if rows is None else np.unique(np.concatenate([[0, n - 1, n // 2], rng.integers(0, n, rows)]))
        for i in some if rows is not None else [0]:
            at = slice(cu[b], cu[b + 1]) if rows is None else slice(cu[b] + i, cu[b] + i + 1)
            kk = slice(cu_k[b], max(cu_k[b], cu_k[b + 1]))
            want, want_lse, tol, ltol = gr.attend(ref.f64(q[at]), ref.f64(k[kk]), ref.f64(v[kk]), past + i, FOREVER if window is None else window,
                                                  sinks, d ** -0.5 if scale is None else scale)
            g, gl = ref.f64(got[at]), lse[at]
            empty = np.isneginf(want_lse)
            assert (np.isneginf(gl) == empty).all() and (g[empty] == 0).all(), (b, i)
            assert (np.abs(gl[~empty] - want_lse[~empty]) <= ltol[~empty]).all(), (b, i)
            assert (np.abs(g - want) <= tol).all(), (b, i, np.abs(g - want).max())


@pytest.mark.parametrize("lens,pasts,H,K,d,window,sink", [
    ([1], [0], 1, 1, 16, None, False), ([37], [0], 32, 8, 128, None, False), ([5, 0, 17, 1, 130], [0, 0, 0, 0, 0], 8, 8, 64, None, True),
    ([64, 65, 127, 128, 129], [0] * 5, 4, 2, 96, None, False), ([200, 3], [0, 300], 20, 4, 128, None, True), ([257], [131], 6, 2, 64, 100, False),
    ([150, 150], [0, 40], 5, 1, 80, 1, True), ([20, 9], [5, 0], 4, 4, 32, 0, True), ([300], [0], 12, 4, 48, 33, True), ([40, 33], [0, 700], 128, 1, 64, 200, False),
    ([9, 100], [1000, 513], 14, 2, 112, None, False), ([1, 1, 1], [0, 127, 128], 64, 8, 128, None, True), ([31], [7], 96, 1, 128, None, False),
    ([70], [-30], 8, 2, 64, None, True), ([10, 200], [-10, -200], 4, 1, 128, None, False)])
def test_matches_formula(torch_dev, lens, pasts, H, K, d, window, sink):
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(H + d + len(lens)), lens, pasts, H, K, d, window, sink)


@pytest.mark.parametrize("lens,pasts,H,K,d,window", [
    ([1500, 613], [0, 0], 8, 2, 128, None), ([2100], [333], 4, 4, 64, 777), ([900, 1, 1300], [0, 5000, 2], 16, 2, 96, None)])
def test_long_prompts_at_some_rows(torch_dev, lens, pasts, H, K, d, window):
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(d), lens, pasts, H, K, d, window, True, rows=9)


def test_padded_batch_no_offsets_and_scales(torch_dev):
    torch, dev = torch_dev
    check(torch, dev, np.random.default_rng(1), [30, 70], [0, 10], 8, 2, 64, pad=7)
    check(torch, dev, np.random.default_rng(2), [140], [0], 8, 2, 128, offsets=False)
    check(torch, dev, np.random.default_rng(3), [140], [0], 8, 2, 128, scale=3.0)
    check(torch, dev, np.random.default_rng(4), [140], [0], 8, 2, 128, size=1e20, scale=1e-20)


def test_scores_that_rise_by_thousands(torch_dev):
    """Keys of growing size: the running maximum moves at every tile."""
    torch, dev = torch_dev
    rng = np.random.default_rng(5)
    n, H, K, d = 600, 4, 2, 64
    q = ref.bf16(np.abs(rng.standard_normal((n, H, d))))
    k = ref.bf16(np.abs(rng.standard_normal((n, K, d))) * np.linspace(0.1, 40, n)[:, None, None])
    v = ref.bf16(rng.standard_normal((n, K, d)))
    got, lse, cu, _ = call(torch, dev, q, k, v, [n], [0], None, None, None, 0)
    want, want_lse, tol, ltol = gr.attend(ref.f64(q), ref.f64(k), ref.f64(v), 0, FOREVER, None, d ** -0.5)
    assert (np.abs(ref.f64(got) - want) <= tol).all() and (np.abs(lse - want_lse) <= ltol).all()


def test_large_values_under_rising_scores(torch_dev):
    """Values of 10^30 while the scores rise from key to key: no product leaves fp32's range."""
    torch, dev = torch_dev
    rng = np.random.default_rng(15)
    n, H, K, d = 500, 4, 2, 128
    q = ref.bf16(np.abs(rng.standard_normal((n, H, d))))
    k = ref.bf16(np.abs(rng.standard_normal((n, K, d))) * np.linspace(0.05, 6, n)[:, None, None])
    v = ref.bf16(1e30 * rng.standard_normal((n, K, d)))
    got, lse, cu, _ = call(torch, dev, q, k, v, [n], [0], None, None, None, 0)
    want, want_lse, tol, ltol = gr.attend(ref.f64(q), ref.f64(k), ref.f64(v), 0, FOREVER, None, d ** -0.5)
    assert (np.abs(ref.f64(got) - want) <= tol).all() and (np.abs(lse - want_lse) <= ltol).all()


@pytest.mark.parametrize("G", [1, 3, 8])
def test_infinities_and_nan_reach_only_the_queries_that_see_them(torch_dev, G):
    """A token's bad values and keys show in its own and later rows of its sequence, within the window, and nowhere else."""
    torch, dev = torch_dev
    K, d, lens, window = 2, 64, [150, 90, 200], 60
    H, rng = K * G, np.random.default_rng(6 + G)
    T = sum(lens)
    q, k, v = ref.bf16(rng.standard_normal((T, H, d))), ref.bf16(rng.standard_normal((T, K, d))), ref.bf16(rng.standard_normal((T, K, d)))
    bad_v, bad_k = [(100, 0, 3, 0x7FC0), (149, 1, 7, 0x7F80), (150 + 40, 0, 9, 0xFF80), (240, 1, 63, 0x7FC0), (439, 0, 0, 0x7F80)], (300, 1)
    for w in (None, window):
        vb, kb = v.copy(), k.copy()
        for t, h, e, bits in bad_v:
            vb[t, h, e] = bits
        kb[bad_k[0], bad_k[1]] = 0x7FC0
        got, lse, cu, _ = call(torch, dev, q, kb, vb, lens, [0, 0, 0], w, None, None, 0)
        f = ref.f64(got)
        bad = np.zeros(f.shape, bool)
        seq = np.repeat(np.arange(3), lens)
        reach = lambda t: [r for r in range(t, T) if seq[r] == seq[t] and (w is None or r - t < w)]
        for t, h, e, _ in bad_v:
            bad[np.ix_(reach(t), range(h * G, (h + 1) * G), [e])] = True
        bad[np.ix_(reach(bad_k[0]), range(bad_k[1] * G, (bad_k[1] + 1) * G))] = True
        assert (np.isfinite(f) == ~bad).all()
        clean = call(torch, dev, q, k, v, lens, [0, 0, 0], w, None, None, 0)[0]
        assert np.abs(f - ref.f64(clean))[~bad].max() <= 2.0 ** -7 * np.abs(ref.f64(clean)).max()
        # an infinity keeps its sign
        assert (f[149, G:2 * G, 7] == np.inf).all() and (f[190, :G, 9] == -np.inf).all() and (f[439, :G, 0] == np.inf).all()


def test_every_key_counts_once(torch_dev):
    """Equal weights and one value that differs: no key is lost or doubled at a tile's border."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    n, H, K, d = 700, 8, 2, 64
    q = torch.randn((n, H, d), device=dev).bfloat16()
    k = torch.zeros((n, K, d), dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    out, lse = torch.empty_like(q), torch.empty((n, H), device=dev)
    i = np.arange(n)
    for j in [0, 1, 63, 64, 127, 128, 129, 255, 256, 300, 383, 384, 500, 511, 512, 640, 699]:
        v.zero_()
        v[j] = 4.0
        fm.fm_prompt_attn(q, k, v, out, lse_out=lse)
        want = np.where(i >= j, 4.0 / (i + 1), 0.0)[:, None, None]
        assert (np.abs(out.double().cpu().numpy() - want) <= want * (2.0 ** -7 + 2.0 ** -12)).all(), j
    assert np.abs(lse.double().cpu().numpy() - np.log(i + 1)[:, None]).max() <= 2.0 ** -19


def test_graph_and_streams_give_the_same_bits(torch_dev):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    lens = torch.tensor([0, 400, 401, 900], dtype=torch.int32, device=dev)
    q, k, v = (torch.randn((900, h, 128), device=dev).bfloat16() for h in (8, 2, 2))
    want, lse = torch.empty_like(q), torch.empty((900, 8), device=dev)
    fm.fm_prompt_attn(q, k, v, want, cu_q=lens, lse_out=lse)
    side, g, out = torch.cuda.Stream(dev), torch.cuda.CUDAGraph(), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        fm.fm_prompt_attn(q, k, v, out, cu_q=lens)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        other = torch.empty_like(q)
        with torch.cuda.stream(side):
            g.replay()
        fm.fm_prompt_attn(q, k, v, other, cu_q=lens)
        torch.cuda.synchronize()
        assert (out.view(torch.int16) == want.view(torch.int16)).all() and (other.view(torch.int16) == want.view(torch.int16)).all()
    assert fm.fm_device_status(reset=True) == 0


@pytest.mark.parametrize("G,d", [(3, 64), (5, 64), (5, 128), (7, 128), (9, 64), (24, 128)])
def test_other_rows_of_a_tile_have_no_part_in_a_sequences_bits(torch_dev, G, d):
    """A sequence alone, before another one of large queries, before rows behind the last sequence, and after a call that left
    large numbers in shared memory: the same bits."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    K, n, past, other = 2, 50, 700, 77
    H, rng = K * G, np.random.default_rng(G + d)
    q, k, v = (up(torch, dev, ref.bf16(rng.standard_normal(s)).view(np.int16)) for s in ((n, H, d), (n + past, K, d), (n + past, K, d)))
    large, zero = up(torch, dev, ref.bf16(60 * rng.standard_normal((other, H, d))).view(np.int16)), torch.zeros((other, H, d), dtype=torch.int16, device=dev)
    full = [up(torch, dev, ref.bf16(60 * rng.standard_normal((38912, 1, d))).view(np.int16)), torch.zeros((38912, 1, d), dtype=torch.int16, device=dev)]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    kv = torch.zeros((other, K, d), dtype=torch.int16, device=dev)
    results = []
    for behind in (None, large, zero):
        for sequences in ((1,) if behind is None else (1, 2)):
            for before in full:  # a tile of 128 tokens of one head: every row of Q's shared memory
                fm.fm_prompt_attn(before, full[1][:128], full[1][:128], torch.empty_like(before), cu_q=i32(0, 38912), cu_k=i32(0, 128), window=1)
                qq = q if behind is None else torch.cat([q, behind])
                kk, vv = (x if behind is None else torch.cat([x, kv]) for x in (k, v))
                ends = ((0, n), (0, n + past)) if sequences == 1 else ((0, n, n + other), (0, n + past, n + past + other))
                out, lse = torch.empty_like(qq), torch.empty(qq.shape[:2], device=dev)
                fm.fm_prompt_attn(qq, kk, vv, out, cu_q=i32(*ends[0]), cu_k=i32(*ends[1]), lse_out=lse)
                results.append((out[:n].clone(), lse[:n].clone()))
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    for out, lse in results[1:]:
        assert (out == results[0][0]).all().item() and (lse == results[0][1]).all().item()
    want, _, tol, _ = gr.attend(ref.f64(q.cpu().numpy().view(np.uint16)), ref.f64(k.cpu().numpy().view(np.uint16)),
                                ref.f64(v.cpu().numpy().view(np.uint16)), past, FOREVER, None, d ** -0.5)
    assert (np.abs(ref.f64(results[0][0].cpu().numpy().view(np.uint16)) - want) <= tol).all()


@pytest.mark.parametrize("size", [100.0, 600.0])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 5)])
def test_scores_of_millions(torch_dev, size, d, G):
    """Scores of up to 2^23, whose spacing in fp32 is coarse: out is finite and a mean of the values whose scores may be the
    largest."""
    torch, dev = torch_dev
    K, n, rng = 2, 300, np.random.default_rng(int(np.log2(size)) + d)
    q, k, v = ref.bf16(size * rng.standard_normal((n, K * G, d))), ref.bf16(size * rng.standard_normal((n, K, d))), ref.bf16(rng.standard_normal((n, K, d)))
    got, lse, _, _ = call(torch, dev, q, k, v, [n], [0], None, None, None, 0)
    f, qf, kf, vf = ref.f64(got), ref.f64(q), ref.f64(k), ref.f64(v)
    assert np.isfinite(f).all()
    for h in range(K * G):
        score = qf[:, h] @ kf[:, h // G].T * d ** -0.5
        score[np.triu_indices(n, 1)] = -np.inf
        bound = ((d + 8) * 2.0 ** -23 * (np.abs(qf[:, h]) @ np.abs(kf[:, h // G]).T) * d ** -0.5 * np.tri(n)).max(1)
        top = score.max(1)
        assert (np.abs(lse[:, h] - top) <= bound + np.log(n) + 2.0 ** -21 * np.abs(top)).all()
        for i in range(n):
            x = vf[score[i] >= top[i] - 2 * bound[i] - 20, h // G]
            slack = 2.0 ** -6 * np.abs(vf[:, h // G]).max(0)
            assert (f[i, h] >= x.min(0) - slack).all() and (f[i, h] <= x.max(0) + slack).all(), (h, i)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 5)])
def test_a_sink_far_over_the_scores(torch_dev, d, G):
    """A sink 60 to 100 nats over every score: the output is as much smaller, to the end of fp32's range, and lse is unchanged."""
    torch, dev = torch_dev
    K, n, rng = 2, 300, np.random.default_rng(d)
    q, k, v = (ref.bf16(rng.standard_normal(s)) for s in ((n, K * G, d), (n, K, d), (n, K, d)))
    for over in (60.0, 88.0, 95.0, np.inf):
        sinks = np.full(K * G, over, np.float32)
        got, lse, _, _ = call(torch, dev, q, k, v, [n], [0], None, sinks, None, 0)
        want, want_lse, tol, ltol = gr.attend(ref.f64(q), ref.f64(k), ref.f64(v) * 2.0 ** 60, 0, FOREVER, sinks, d ** -0.5)
        # grouped_ref's absolute term of 2^-120 is these outputs' size, so values are 2^60 times as large there; a step of
        # bf16's subnormals; an exponential of an argument of 100 is off by 2^-16
        assert (np.abs(ref.f64(got) * 2.0 ** 60 - want) <= tol + 2.0 ** -15 * np.abs(want) + 2.0 ** (60 - 133)).all(), over
        assert (np.abs(lse - want_lse) <= ltol).all()
