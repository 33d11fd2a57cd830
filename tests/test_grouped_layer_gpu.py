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
