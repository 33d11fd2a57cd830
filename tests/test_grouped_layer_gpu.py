"""The calls of a dense layer of grouped heads together, as a model's prompt and decode steps make them: norm and
rotation, the prompt's attention, its keys and values into the 8-bit cache, then steps of one and of
several tokens over the cache."""
import numpy as np
import pytest

import attn_ref as ref
import grouped_ref as gr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


@pytest.mark.parametrize("d,H,K,rope", [(128, 8, 2, 64), (96, 6, 2, 96), (64, 5, 1, 0)])
def test_prompt_then_decode(torch_dev, d, H, K, rope):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    g = torch.Generator(device=dev).manual_seed(d)
    prompts, steps = [70, 1, 33], [1, 1, 3, 1]
    B = len(prompts)
    i32 = lambda a: torch.tensor(np.array(a), dtype=torch.int32, device=dev)
    R = (max(prompts) + sum(steps) + 63) // 64
    P = B * R
    table = torch.randperm(P, generator=g, device=dev).int().view(B, R)
    pool = torch.full((2, P, K, 64, d), 0x7F, dtype=torch.uint8, device=dev)
    scale = torch.full((2, P, K, 4), float("nan"), device=dev)
    seen = [[np.zeros((0, K, d)), np.zeros((0, K, d))] for _ in range(B)]  # what each sequence's cache should hold
    have = [0] * B
    for step, ns in enumerate([prompts] + [[n] * B for n in steps]):
        T = sum(ns)
        cu = np.concatenate([[0], np.cumsum(ns)])
        x = torch.randn((T, (H + 2 * K) * d), generator=g, device=dev).bfloat16()
        q, k, v = x[:, :H * d].view(T, H, d), x[:, H * d:(H + K) * d].view(T, K, d), x[:, (H + K) * d:].view(T, K, d)
        start = torch.tensor(have, dtype=torch.int64, device=dev)
        pos = torch.cat([torch.arange(h, h + n, device=dev) for h, n in zip(have, ns)])
        # norm and rotation of queries and keys in one call; the cache then takes the keys as they are
        qn, kn, out = torch.empty((T, H, d), dtype=torch.bfloat16, device=dev), torch.empty((T, K, d), dtype=torch.bfloat16, device=dev), None
        fm.fm_qk_norm_rope(pos, q=q, q_out=qn, k=k, k_out=kn, rope_dim=rope)
        out = torch.empty_like(qn)
        fm.fm_kv_append_fp8(kn, v, pool[0], pool[1], scale[0], scale[1], table, start, cu_tokens=i32(cu), rope_dim=0)
        if step == 0:
            fm.fm_prompt_attn(qn, kn, v, out, cu_q=i32(cu))
        else:
            ws = torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(T, H, K, d)), dtype=torch.uint8, device=dev)
            fm.fm_kv_attn_fp8(qn, pool[0], pool[1], scale[0], scale[1], table, start, out, cu_tokens=i32(cu), workspace=ws)
        torch.cuda.synchronize()
        assert fm.fm_device_status(reset=True) == 0
        kf, vf, qf, of = (t.double().cpu().numpy() for t in (kn, v, qn, out))
        codes, scales = gr.VALUES[pool.cpu().numpy()], scale.double().cpu().numpy()
        for b in range(B):
            rows = slice(cu[b], cu[b + 1])
            for i, y in ((0, kf), (1, vf)):
                seen[b][i] = np.concatenate([seen[b][i], y[rows]])
            m = have[b] + ns[b]
            j = np.arange(m)
            page = table[b].cpu().numpy()[j // 64]
            cached = [codes[i][page, :, j % 64] * scales[i][page, :, j % 64 // 16][..., None] for i in (0, 1)]
            for i in (0, 1):  # E4M3 with a scale of the block's largest: half a step of the value or of the block's subnormals
                block = np.stack([np.abs(seen[b][i][lo:lo + 16]).max((0, 2)) for lo in range(0, m, 16)])[j // 16][..., None]
                # a block that grew was rounded again at each new scale: up to one more half step
                assert (np.abs(cached[i] - seen[b][i]) <= 2 * (2.0 ** -4 * np.abs(seen[b][i]) + 2.0 ** -9 * block / 224)).all()
            if step == 0:
                want, _, tol, _ = gr.attend(qf[rows], kf[rows], vf[rows], 0, 1 << 60, None, d ** -0.5)
            else:
                size = np.abs(codes[1][page, :, j % 64])
                want, _, tol, _ = gr.attend(qf[rows], cached[0], cached[1], have[b], 1 << 60, None, d ** -0.5, None, gr.HALF_FP16,
                                            (size, scales[1][page, :, j % 64 // 16][..., None]))
            assert (np.abs(of[rows] - want) <= tol).all(), (step, b)
        have = [h + n for h, n in zip(have, ns)]
    assert (pool.cpu().numpy()[1] != 0x7F).any()


def test_the_append_turns_what_the_norm_would(torch_dev):
    """A model without a norm lets the append turn keys and queries: the cells and queries are those of the turned tensors
    of the formula, and the decode step over them matches it."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    g = torch.Generator(device=dev).manual_seed(3)
    B, H, K, d, have = 4, 8, 2, 64, [0, 15, 64, 200]
    R = 4
    table = torch.randperm(B * R, generator=g, device=dev).int().view(B, R)
    pool = torch.zeros((2, B * R, K, 64, d), dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.ones((2, B * R, K, 4), device=dev)
    out = torch.empty((B, H, d), dtype=torch.bfloat16, device=dev)
    q, q_out = torch.randn((B, H, d), generator=g, device=dev).bfloat16(), torch.empty((B, H, d), dtype=torch.bfloat16, device=dev)
    k, v = (torch.randn((B, K, d), generator=g, device=dev).bfloat16() for _ in "kv")
    start = torch.tensor(have, device=dev)
    fm.fm_kv_append_fp8(k, v, pool[0], pool[1], scale[0], scale[1], table, start, q=q, q_out=q_out)
    ws = torch.empty(max(1, fm.fm_kv_attn_fp8_workspace(B, H, K, d)), dtype=torch.uint8, device=dev)
    fm.fm_kv_attn_fp8(q_out, pool[0], pool[1], scale[0], scale[1], table, start, out, window=1, workspace=ws)
    torch.cuda.synchronize()
    turned = gr.rotate(k.double().cpu().numpy(), np.array(have), 64)
    codes, scales = pool.double().cpu().numpy(), scale.double().cpu().numpy()
    for b, h in enumerate(have):
        page, row = int(table[b, h // 64]), h % 64
        got_k = codes[0][page, :, row] * scales[0][page, :, row // 16, None]
        got_v = codes[1][page, :, row] * scales[1][page, :, row // 16, None]
        near = lambda x: 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * max(1.0, np.abs(x).max()) / 224 + 2.0 ** -9 * scales.max()
        assert (np.abs(got_k - turned[b]) <= near(turned[b])).all()
        # one key: the output is its value
        want = np.repeat(got_v, H // K, 0)
        assert (np.abs(out[b].double().cpu().numpy() - want) <= 2.0 ** -7 * np.abs(want)).all()


def test_offsets_past_32_bits(torch_dev):
    """A layer among a thousand: its pages are 16 MB apart, the last ones past 2^32 bytes."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    H, K, d, L, P = 4, 2, 128, 1024, 300
    pools = [torch.zeros((P, L, K, 64, d), dtype=torch.uint8, device=dev) for _ in "kv"]
    scales = [torch.ones((P, L, K, 4), device=dev) for _ in "kv"]
    assert pools[0].numel() > 1 << 32
    (kp, vp), (ks, vs) = ([t[:, 1000] for t in x] for x in (pools, scales))
    table = torch.tensor([[299, 0, 298]], dtype=torch.int32, device=dev)
    n = 150
    g = torch.Generator(device=dev).manual_seed(1)
    q, k, v = (torch.randn((n, h, d), generator=g, device=dev).bfloat16() for h in (H, K, K))
    cu, start = torch.tensor([0, n], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
    fm.fm_kv_append_fp8(k, v, kp, vp, ks, vs, table, start, cu_tokens=cu, rope_dim=0)
    out = torch.empty((1, H, d), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(1, H, K, d), dtype=torch.uint8, device=dev)
    fm.fm_kv_attn_fp8(q[-1:].contiguous(), kp, vp, ks, vs, table, start + n - 1, out, workspace=ws)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    assert all(int(p[:, :1000].sum()) == 0 and int(p[:, 1001:].sum()) == 0 for p in pools)
    codes = np.stack([gr.VALUES[x.cpu().numpy()] for x in (kp, vp)])
    sc = np.stack([x.double().cpu().numpy() for x in (ks, vs)])
    j = np.arange(n)
    page = table[0].cpu().numpy()[j // 64]
    cells = [codes[i][page, :, j % 64] * sc[i][page, :, j % 64 // 16][..., None] for i in (0, 1)]
    for i, x in ((0, k), (1, v)):
        x = x.double().cpu().numpy()
        block = np.stack([np.abs(x[lo:lo + 16]).max((0, 2)) for lo in range(0, n, 16)])[j // 16][..., None]
        assert (np.abs(cells[i] - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * block / 224).all()
    want, _, tol, _ = gr.attend(q[-1:].double().cpu().numpy(), cells[0], cells[1], n - 1, 1 << 60, None, d ** -0.5, None, gr.HALF_FP16,
                                (np.abs(codes[1][page, :, j % 64]), sc[1][page, :, j % 64 // 16][..., None]))
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_arguments_on_their_own_borders_only(torch_dev):
    """Every tensor begins 16 bytes (or one element, where that is allowed) into a larger one, and rows lie apart."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    n, H, K, d = 70, 6, 3, 80
    g = torch.Generator(device=dev).manual_seed(2)

    def inside(t, skip):
        flat = torch.zeros(t.numel() + 64, dtype=t.dtype, device=dev)[skip:skip + t.numel()].view(t.shape)
        return flat.copy_(t)
    rows = lambda h: torch.randn((n, h * d + 24), generator=g, device=dev).bfloat16()[:, 8:8 + h * d].unflatten(1, (h, d))
    q, k, v = rows(H), rows(K), rows(K)
    ints = lambda x, t: inside(torch.tensor(x, dtype=t, device=dev), 1)
    cu, table, start = ints([0, 30, n], torch.int32), ints([[1, 3], [0, 2]], torch.int32), ints([0, 9], torch.int64)
    pool = [inside(torch.zeros((4, K, 64, d), dtype=torch.uint8, device=dev), 16) for _ in "kv"]
    scale = [inside(torch.ones((4, K, 4), device=dev), 4) for _ in "kv"]
    sink, lse, lse2 = ints([0.5] * H, torch.float32), inside(torch.zeros((n, H), device=dev), 1), inside(torch.zeros((n, H), device=dev), 3)
    out, out2 = (inside(torch.zeros((n, H, d), dtype=torch.bfloat16, device=dev), 8) for _ in "ab")
    fm.fm_kv_append_fp8(k, v, *pool, *scale, table, start, cu_tokens=cu, rope_dim=0)
    ws = torch.empty(fm.fm_kv_attn_fp8_workspace(n, H, K, d), dtype=torch.uint8, device=dev)
    fm.fm_kv_attn_fp8(q, *pool, *scale, table, start, out, cu_tokens=cu, window=20, sink_logit=sink, lse_out=lse, workspace=ws)
    fm.fm_prompt_attn(q, k, v, out2, cu_q=cu, window=20, sink_logit=sink, lse_out=lse2)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    qf, kf, vf = (t.double().cpu().numpy() for t in (q, k, v))
    for b, (lo, hi) in enumerate(((0, 30), (30, n))):
        want, wl, tol, lt = gr.attend(qf[lo:hi], kf[lo:hi], vf[lo:hi], 0, 20, np.full(H, 0.5), d ** -0.5)
        assert (np.abs(out2[lo:hi].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse2[lo:hi].double().cpu().numpy() - wl) <= lt).all()
        s = int(start[b])
        j = np.arange(s, s + hi - lo)
        page = table[b].cpu().numpy()[j // 64]
        codes = [gr.VALUES[x.cpu().numpy()][page, :, j % 64] for x in pool]
        sc = [x.double().cpu().numpy()[page, :, j % 64 // 16][..., None] for x in scale]
        if s == 0:  # the second sequence's first nine cells were never written: zeros, with weight
            want, wl, tol, lt = gr.attend(qf[lo:hi], codes[0] * sc[0], codes[1] * sc[1], 0, 20, np.full(H, 0.5), d ** -0.5, None, gr.HALF_FP16,
                                          (np.abs(codes[1]), sc[1]))
            assert (np.abs(out[lo:hi].double().cpu().numpy() - want) <= tol).all()
            assert (np.abs(lse[lo:hi].double().cpu().numpy() - wl) <= lt).all()
