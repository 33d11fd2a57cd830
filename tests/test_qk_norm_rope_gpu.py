"""fm_qk_norm_rope against the fp64 formula: widths, strides, positions, cells."""
import numpy as np
import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu
PAGE = ref.PAGE


@pytest.fixture(scope="module")
def torch_dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def up(torch, dev, a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


@pytest.mark.parametrize("T,H,K,d,rope", [
    (1, 64, 1, 512, 64), (3, 1, 1, 8, 8), (7, 5, 2, 64, 64), (2, 128, 8, 128, 64), (5, 3, 1, 96, 50), (4, 9, 4, 200, 0),
    (33, 20, 1, 576, 64), (2, 7, 3, 1024, 256), (1300, 2, 1, 256, 128), (3, 64, 1, 512, 2), (5, 0, 3, 512, 64),
    (5, 3, 0, 512, 64)])
def test_matches_formula(torch_dev, T, H, K, d, rope):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(T + H + d)
    x = ref.bf16(3 * rng.standard_normal((T, (H + K) * d + 24)))  # a fused projection with 24 elements more
    x[T // 2] = 0  # a row of zeros: eps keeps it finite
    qg, kg = ref.bf16(1 + 0.2 * rng.standard_normal(d)), ref.bf16(1 + 0.2 * rng.standard_normal(d))
    pos = rng.integers(0, 1 << 21, T)
    pos[0] = 0
    P = T // PAGE + 2
    cell = rng.permutation(P * PAGE)[:T].astype(np.int32)
    cell[T // 3] = -1 if T > 2 else cell[T // 3]
    old = ref.bf16(rng.standard_normal((P, 2, PAGE, max(K, 1) * d)))
    xd = up(torch, dev, x.view(np.int16))
    q, k = xd[:, :H * d].view(T, H, d), xd[:, H * d:(H + K) * d].view(T, K, d)
    q_out = torch.empty((T, H, d), dtype=torch.int16, device=dev)
    k_out = torch.empty((T, K, d), dtype=torch.int16, device=dev)
    pool = up(torch, dev, old.view(np.int16))
    kw = dict(pos=up(torch, dev, pos), rope_dim=rope, eps=1e-6)
    if H:
        kw.update(q=q, q_gain=up(torch, dev, qg.view(np.int16)), q_out=q_out)
    if K:
        kw.update(k=k, k_gain=None if T == 3 else up(torch, dev, kg.view(np.int16)), k_out=k_out, k_pool=pool[:, 1],
                  k_cell=up(torch, dev, cell))
    fm.fm_qk_norm_rope(**kw)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    xf = ref.f64(x)
    if H:
        want, tol = ref.norm_rope(xf[:, :H * d].reshape(T, H, d), ref.f64(qg), pos, rope, 1e-6)
        got = ref.f64(q_out.cpu().numpy().view(np.uint16))
        assert (np.abs(got - want) <= tol).all()
    if K:
        gain = None if T == 3 else ref.f64(kg)
        want, tol = ref.norm_rope(xf[:, H * d:(H + K) * d].reshape(T, K, d), gain, pos, rope, 1e-6)
        got = k_out.cpu().numpy().view(np.uint16)
        assert (np.abs(ref.f64(got) - want) <= tol).all()
        # the pool's rows are the same bits, and no other row has changed
        new = old.copy()
        for t in range(T):
            if cell[t] >= 0:
                new[cell[t] // PAGE, 1, cell[t] % PAGE] = got[t].reshape(-1)
        assert (pool.cpu().numpy().view(np.uint16) == new).all()


def test_in_place_pool_only_and_range(torch_dev):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(3)
    T, H, d = 70, 6, 512
    x = ref.bf16(rng.standard_normal((T, H, d)))
    pos = np.arange(T) + 1048576 - T
    want, tol = ref.norm_rope(ref.f64(x), None, pos, 64, 1e-5, base=10000.0, factor=1.0)
    kw = dict(rope_base=10000.0, rope_factor=1.0, eps=1e-5)
    q = up(torch, dev, x.view(np.int16))
    fm.fm_qk_norm_rope(up(torch, dev, pos), q=q, q_out=q, **kw)
    torch.cuda.synchronize()
    assert (np.abs(ref.f64(q.cpu().numpy().view(np.uint16)) - want) <= tol).all()
    # keys to the pool alone; a cell at the end of the pool and one far past it are skipped and flagged
    pool = torch.zeros((2, PAGE, H * d), dtype=torch.int16, device=dev)
    cell = np.arange(T, dtype=np.int32)
    cell[5], cell[9] = 2 * PAGE, 2 ** 31 - 1
    fm.fm_qk_norm_rope(up(torch, dev, pos), k=up(torch, dev, x.view(np.int16)), k_pool=pool,
                       k_cell=up(torch, dev, cell), **kw)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == fm.FM_DEVERR_PAGE_RANGE
    got = pool.cpu().numpy().view(np.uint16).reshape(2 * PAGE, H, d)
    keep = np.ones(T, bool)
    keep[[5, 9]] = False
    assert (np.abs(ref.f64(got[:T][keep]) - want[keep]) <= tol[keep]).all()
    assert (got[[5, 9]] == 0).all() and (got[T:] == 0).all()
    fm.fm_qk_norm_rope(torch.empty(0, dtype=torch.int64, device=dev), q=q[:0], q_out=q[:0])


def test_far_positions_and_huge_values(torch_dev):
    """Positions past 2^31 keep their angle; a row of the largest bf16 values
    overflows the fp32 square and becomes zero, as 1 / sqrt(inf) says."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(4)
    pos = np.array([2 ** 31 + 7, 2 ** 20, 3, 10 ** 9], np.int64)
    x = ref.bf16(rng.standard_normal((4, 2, 128)))
    out = torch.empty((4, 2, 128), dtype=torch.int16, device=dev)
    fm.fm_qk_norm_rope(up(torch, dev, pos), q=up(torch, dev, x.view(np.int16)), q_out=out)
    want, tol = ref.norm_rope(ref.f64(x), None, pos, 64, 1e-6)
    # pos * theta is itself formed in fp64 by the formula: off by pos * 2^-52 radians at most
    tol += 2 * (pos * 2.0 ** -52)[:, None, None] * 4
    torch.cuda.synchronize()
    assert (np.abs(ref.f64(out.cpu().numpy().view(np.uint16)) - want) <= tol).all()
    x[:] = 0x7F7F
    fm.fm_qk_norm_rope(up(torch, dev, pos), q=up(torch, dev, x.view(np.int16)), q_out=out, rope_dim=0)
    torch.cuda.synchronize()
    assert (out == 0).all()


def test_graph_replay_takes_new_inputs(torch_dev):
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(5)
    xs = [up(torch, dev, ref.bf16(rng.standard_normal((3, 64, 512))).view(np.int16)) for _ in range(2)]
    pos = up(torch, dev, np.arange(3) + 77)
    x, out = xs[0].clone(), torch.empty_like(xs[0])
    fm.fm_qk_norm_rope(pos, q=x, q_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.fm_qk_norm_rope(pos, q=x, q_out=out)
    x.copy_(xs[1])
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    fm.fm_qk_norm_rope(pos, q=xs[1], q_out=out)
    torch.cuda.synchronize()
    assert torch.equal(got, out)


def test_offsets_past_32_bits_and_most_heads(torch_dev):
    """More than 2^32 elements of queries, and of the pool; the most heads and the
    widest one."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    T, H, K, d = 1060, 4000, 96, 1024
    g = torch.Generator(device=dev).manual_seed(6)
    q = torch.randn((T, H, d), generator=g, device=dev, dtype=torch.bfloat16)
    k = torch.randn((T, K, d), generator=g, device=dev, dtype=torch.bfloat16)
    assert q.numel() > 1 << 32
    P = (1 << 32) // (PAGE * K * d) + 2
    pool = torch.zeros((P, PAGE, K * d), dtype=torch.bfloat16, device=dev)
    pos = torch.arange(T, device=dev) * 997
    cell = (P * PAGE - 1 - torch.arange(T, device=dev)).int()
    out = torch.empty_like(q)
    fm.fm_qk_norm_rope(pos, q=q, q_out=out, k=k, k_pool=pool, k_cell=cell, rope_dim=256)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == 0
    rows = pool.view(P * PAGE, K, d)
    for t in (0, T // 2, T - 1):
        at = np.array([t * 997])
        for x, y in ((q[t], out[t]), (k[t], rows[int(cell[t])])):
            want, tol = ref.norm_rope(x[None].double().cpu().numpy(), None, at, 256, 1e-6)
            assert (np.abs(y[None].double().cpu().numpy() - want) <= tol).all()


def test_many_tokens(torch_dev):
    """More than two million tokens of one narrow head."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    T = (1 << 21) + 5
    x = torch.randn((T, 1, 8), generator=torch.Generator(device=dev).manual_seed(7), device=dev, dtype=torch.bfloat16)
    pos, out = torch.arange(T, device=dev), torch.empty_like(x)
    fm.fm_qk_norm_rope(pos, q=x, q_out=out, rope_dim=8)
    torch.cuda.synchronize()
    want, tol = ref.norm_rope(x.double().cpu().numpy(), None, pos.cpu().numpy(), 8, 1e-6)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
