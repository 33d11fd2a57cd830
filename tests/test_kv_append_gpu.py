"""fm_kv_append_fp8 against the fp64 formula: blocks begun and continued, rotation, scales, pages not held,
strides, padded batches, graphs."""
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


def up(torch, dev, a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def tables(rng, lens, starts, extra=2):
    """A page table that holds, in a random order, the pages from each sequence's first new token on, with room behind
    its end, and the number of pages."""
    R = max((s + n + 63) // 64 for n, s in zip(lens, starts)) + 1
    table, at = np.full((len(lens), R), -1, np.int32), 0
    for b, s in enumerate(starts):
        table[b, s // 64:] = np.arange(at, at + R - s // 64)
        at += R - s // 64
    order = rng.permutation(at + extra).astype(np.int32)
    return np.where(table < 0, -1, order[table]), at + extra


def check_pool(got, before, want, written, exact, size, what):
    """Codes outside the written cells are as before; each new one is the code of a value within `size` of
    the exact one."""
    assert (got[~written] == before[~written]).all(), f"{what}: a cell was written that is not the call's"
    new = ~np.isnan(exact)
    other = written & ~new
    assert (got[other] == want[other]).all(), f"{what}: NaN cells or requantised cells"
    value, z, d = gr.VALUES[got[new]], exact[new], size[new]
    lo, hi = gr.VALUES[gr.e4m3_codes(z - d)], gr.VALUES[gr.e4m3_codes(z + d)]
    assert ((lo <= value) & (value <= hi)).all(), what


def run(torch, dev, rng, lens, starts, K, d, H, rope, k=None, v=None, table=None, P=None, pools=None, scales=None, pad=0, gaps=True,
        flags=0, **yarn):
    import sparse_attention_kv_c4_gb300 as fm
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + pad
    if table is None:
        table, P = tables(rng, lens, starts)
    fused = ref.bf16(2 * rng.standard_normal((T, (H + 2 * K) * d + 8)))
    if k is not None:
        fused[:, H * d:(H + K) * d] = k.reshape(T, -1)
    if v is not None:
        fused[:, (H + K) * d:(H + 2 * K) * d] = v.reshape(T, -1)
    f = up(torch, dev, fused.view(np.int16))
    part = lambda a, b, h: f[:, a * d:b * d].view(T, h, d)
    layers = 3 if gaps else 1  # the layer's pages lie between other layers'
    if pools is None:
        pools = rng.integers(0, 256, (2, P, layers, K, 64, d)).astype(np.uint8)
        pools[(pools & 127) == 127] = 0
        scales = (2.0 ** rng.integers(-4, 3, (2, P, layers, K, 4))).astype(np.float32)
    pd, sd = up(torch, dev, pools), up(torch, dev, scales)
    mid = layers // 2
    q_out = torch.full((T, H, d), 77, dtype=torch.int16, device=dev) if H else None
    fm.fm_kv_append_fp8(part(H, H + K, K), part(H + K, H + 2 * K, K), pd[0][:, mid], pd[1][:, mid], sd[0][:, mid], sd[1][:, mid],
                        up(torch, dev, table), up(torch, dev, np.array(starts, np.int64)), cu_tokens=up(torch, dev, cu),
                        q=part(0, H, H) if H else None, q_out=q_out, rope_dim=rope, **yarn)
    torch.cuda.synchronize()
    assert fm.fm_device_status(reset=True) == flags
    got_p, got_s = pd.cpu().numpy(), sd.cpu().numpy()
    names = dict(base=yarn.get("rope_base", 160000.0), factor=yarn.get("rope_factor", 16.0))
    kf, vf = ref.f64(fused[:, H * d:(H + K) * d]).reshape(T, K, d), ref.f64(fused[:, (H + K) * d:(H + 2 * K) * d]).reshape(T, K, d)
    want_p, want_s = [pools[i][:, mid].copy() for i in (0, 1)], [scales[i][:, mid].copy() for i in (0, 1)]
    written, exact = gr.append(kf, vf, want_p, want_s, table, starts, cu, rope, **names)
    for i, what in ((0, "keys"), (1, "values")):
        assert np.array_equal(got_s[i][:, mid], want_s[i]), f"{what}: scales"
        assert (np.delete(got_p[i], mid, 1) == np.delete(pools[i], mid, 1)).all()
        assert (np.delete(got_s[i], mid, 1) == np.delete(scales[i], mid, 1)).all()
        # rotation in fp32: an angle good to 2^-23, its sine and cosine, two products and a sum: 2^-20 of the pair
        size = np.zeros(exact[i].shape)
        if i == 0 and rope:
            e = exact[i][..., d - rope:]
            pair = np.sqrt(e[..., 0::2] ** 2 + e[..., 1::2] ** 2)
            size[..., d - rope:] = np.repeat(np.nan_to_num(pair), 2, -1) * 2.0 ** -20
        check_pool(got_p[i][:, mid], pools[i][:, mid], want_p[i], written[i], exact[i], size, what)
    if H:
        pos = np.concatenate([s + np.arange(n) for n, s in zip(lens, starts)] + [np.zeros(pad, np.int64)])
        qf = ref.f64(fused[:, :H * d]).reshape(T, H, d)
        want = gr.rotate(qf, pos, rope, **names)
        pair = np.zeros_like(want)
        if rope:
            a = want[..., d - rope:]
            pair[..., d - rope:] = np.repeat(np.sqrt(a[..., 0::2] ** 2 + a[..., 1::2] ** 2), 2, -1)
        got = q_out.cpu().numpy().view(np.uint16)
        live = np.concatenate([np.full(n, s >= 0) for n, s in zip(lens, starts)] + [np.zeros(pad, bool)])
        assert (np.abs(ref.f64(got) - want) <= 2.0 ** -20 * pair + gr.HALF_BF16 * np.abs(want))[live].all()
        assert (got[~live] == 77).all()
        assert (got[..., :d - rope] == fused[:, :H * d].reshape(T, H, d)[..., :d - rope])[live].all()
    return got_p, got_s, table


@pytest.mark.parametrize("lens,starts,K,d,H,rope,pad", [
    ([1], [0], 1, 16, 0, 0, 0), ([1], [1048575], 8, 128, 32, 64, 0), ([1] * 76, [(b * 37) % 200 for b in range(76)], 4, 64, 8, 64, 0),
    ([5, 0, 17, 1, 0, 33], [3, 9, 16, 63, 5, 120], 2, 96, 6, 50, 3), ([200], [7], 3, 128, 3, 128, 5), ([16, 15, 31], [0, 1, 15], 5, 48, 10, 2, 0),
    ([613, 600, 1], [0, 37, 64], 4, 80, 20, 64, 0), ([3] * 40, list(range(40)), 1, 128, 128, 64, 1), ([64, 64], [64, 128], 16, 112, 0, 112, 0),
    ([1] * 1100, [b % 91 for b in range(1100)], 1, 16, 1, 16, 0)])
def test_matches_formula(torch_dev, lens, starts, K, d, H, rope, pad):
    torch, dev = torch_dev
    run(torch, dev, np.random.default_rng(len(lens) + d + H), lens, starts, K, d, H, rope, pad=pad)


def test_plain_rotary_embedding_and_far_positions(torch_dev):
    torch, dev = torch_dev
    run(torch, dev, np.random.default_rng(2), [4, 9], [(1 << 20) - 5, 70000], 2, 64, 4, 64, rope_base=10000.0, rope_factor=1.0)


def test_values_at_the_ends_of_the_types(torch_dev):
    """Zeros, subnormals, the largest finite numbers, infinities and NaN; a row of nothing else."""
    torch, dev = torch_dev
    rng = np.random.default_rng(4)
    T, K, d = 40, 2, 32
    v = ref.bf16(rng.standard_normal((T, K, d)) * 2.0 ** rng.integers(-20, 20, (T, 1, 1)))
    v[0:16] = 0
    v[17, 0, 3:7] = [0x7F80, 0xFF80, 0x7FC0, 0xFFC0]   # +-inf, NaN
    v[32:48] = 0x7FC0                                  # nothing finite in the block
    v[20, 1, :4] = [0x7F7F, 0xFF7F, 0x0001, 0x8001]    # largest and smallest
    v[33, 1, 0] = 0x0001
    got, s, table = run(torch, dev, rng, [T], [0], K, d, 0, 0, v=v, k=v[::-1].copy())
    page = table[0, 0]
    assert (s[1][page, 1, 0, 0] == 2.0 ** -100) and (got[1][page, 1, 0, :16] == 0).all()
    assert (got[1][page, 1, 0, 17, 3:7] & 127 == 127).all()


def test_a_block_filled_token_by_token(torch_dev):
    """Growing magnitudes: each step may raise the block's scale and bring the earlier codes to it; every step
    is the reference's step from the same cache."""
    torch, dev = torch_dev
    rng = np.random.default_rng(6)
    B, K, d = 3, 2, 64
    table, P = tables(rng, [40] * B, [0] * B)
    pools, scales = np.zeros((2, P, 1, K, 64, d), np.uint8), np.ones((2, P, 1, K, 4), np.float32)
    for step in range(20):
        grow = [2.0 ** (step % 7), 2.0 ** (-step), 1.0]
        x = ref.bf16(rng.standard_normal((B, K, d)) * np.array(grow)[:, None, None])
        pools, scales, _ = run(torch, dev, rng, [1] * B, [step + 11 * b for b in range(B)], K, d, 0, 64, k=x, v=x, table=table, P=P,
                               pools=pools, scales=scales, gaps=False)


def test_scales_that_are_no_powers_of_two(torch_dev):
    """A cache of another writer: a continued block keeps a scale that is large enough, and the new entries are
    x * (1 / scale) rounded once from fp32."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(8)
    K, d = 2, 64
    x = ref.bf16(rng.standard_normal((3, K, d)))
    pool = torch.zeros((2, 1, K, 64, d), dtype=torch.uint8, device=dev)
    scale = torch.full((2, 1, K, 4), 0.013, dtype=torch.float32, device=dev)
    xd = up(torch, dev, x.view(np.int16))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    fm.fm_kv_append_fp8(xd, xd, pool[0], pool[1], scale[0], scale[1], i32([[0]]), torch.tensor([5], device=dev), cu_tokens=i32([0, 3]), rope_dim=0)
    inv = np.float32(1) / np.float32(0.013)
    z = (ref.f64(x).astype(np.float32) * inv).astype(np.float64)
    assert (pool[1, 0, :, 5:8].cpu().numpy().transpose(1, 0, 2) == gr.e4m3_codes(z)).all()
    assert (scale == np.float32(0.013)).all().item() and fm.fm_device_status(reset=True) == 0


def test_pages_not_held_and_out_of_range(torch_dev):
    torch, dev = torch_dev
    rng = np.random.default_rng(9)
    lens, starts = [100, 5, 20, 1, 3], [60, 0, 300, -1, 0]
    table, P = np.full((5, 3), -1, np.int32), 9
    table[0] = [4, -1, 6]          # the middle page is not held
    table[1] = [9, 0, 0]           # past the pool: left out and flagged
    table[2] = [1, 2, 3]           # tokens past the table: left out and flagged
    table[3] = [0, 0, 0]           # a negative start: left out, queries too
    table[4] = [8, 7, 5]
    run(torch, dev, rng, lens, starts, 2, 64, 2, 64, table=table, P=P, flags=1)
    table[1], starts[2] = [-1, 0, 0], 0
    run(torch, dev, rng, lens, starts, 2, 64, 2, 64, table=table, P=P)


def test_no_offsets_in_place_queries_streams_and_graph(torch_dev):
    """Without cu_tokens each row is a sequence; q_out may be q; the call is captured and replayed on a
    stream of its own with new inputs in the same buffers."""
    torch, dev = torch_dev
    import sparse_attention_kv_c4_gb300 as fm
    rng = np.random.default_rng(10)
    B, K, d, H = 6, 2, 64, 4
    table, P = tables(rng, [1] * B, [9 * b for b in range(B)])
    pool = torch.zeros((2, P, K, 64, d), dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.ones((2, P, K, 4), device=dev)
    x = torch.randn((B, 2 * K, d), device=dev).bfloat16()
    q = torch.randn((B, H, d), device=dev).bfloat16()
    start = torch.tensor([9 * b for b in range(B)], device=dev)
    td = up(torch, dev, table)
    call = lambda qq, stream=None: fm.fm_kv_append_fp8(x[:, :K], x[:, K:], pool[0], pool[1], scale[0], scale[1], td, start, q=qq,
                                                       q_out=qq, stream=stream)
    side, graph = torch.cuda.Stream(dev), torch.cuda.CUDAGraph()
    q_graph = q.clone()
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.graph(graph, stream=side):
        call(q_graph)
    x.copy_(torch.randn((B, 2 * K, d), device=dev).bfloat16())
    start += 3
    graph.replay()
    torch.cuda.synchronize()
    by_graph, scale_graph = pool.view(torch.uint8).clone(), scale.clone()
    pool.view(torch.uint8).zero_()
    scale.fill_(1)
    q_plain = q.clone()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream(dev))
        call(q_plain)
    torch.cuda.synchronize()
    assert (pool.view(torch.uint8) == by_graph).all() and (scale == scale_graph).all() and (q_plain == q_graph).all()
    assert by_graph.any() and not (q_plain == q).all()
    pos = start.cpu().numpy()
    want = gr.rotate(q.double().cpu().numpy(), pos, 64)
    assert (np.abs(q_plain.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17).all()


@pytest.mark.parametrize("inside,d,K", [(0, 64, 1), (5, 64, 1), (0, 96, 2), (5, 128, 1)])
def test_a_turned_pair_at_the_border_of_a_scale(torch_dev, inside, d, K):
    """Pairs whose larger turned entry lies within 2^-24 of 448 times a power of two, on either side: fp32's rounding of the turn
    would put some on the other side, and with it all of their block's codes."""
    torch, dev = torch_dev
    rope = 64
    pos = 16 * np.arange(0, 256) + inside
    angle = pos[:, None] * ref.freqs(rope)[None, :]
    c, s = np.cos(angle)[..., None], np.sin(angle)[..., None]
    a = (128 + np.arange(128)) / 128.0 * np.ones(c.shape)
    border = 1.75
    with np.errstate(divide="ignore", invalid="ignore"):
        b = ref.f64(ref.bf16((a * c - border) / s))
        x, y = a * c - b * s, a * s + b * c
        near = np.abs(x / border - 1)
    # farther than fp64's own errors, and the larger of the two
    t, i, j = np.nonzero((near < 2.0 ** -24) & (near > 1e-10) & (np.abs(y) < 1.5))
    assert len(t) >= 32 and (x[t, i, j] > border).any() and (x[t, i, j] < border).any()
    T = len(t)
    rng = np.random.default_rng(5)
    k = ref.bf16(0.1 * rng.standard_normal((T, K, d)))
    at = np.arange(T)
    k[at, K - 1, d - rope + 2 * i], k[at, K - 1, d - rope + 2 * i + 1] = ref.bf16(a[t, i, j]), ref.bf16(b[t, i, j])
    starts = [int(p) for p in pos[t]]
    table, at = np.full((T, max(starts) // 64 + 1), -1, np.int32), np.arange(T)
    table[at, np.array(starts) // 64] = at
    pools, scales = np.zeros((2, T, 1, K, 64, d), np.uint8), np.full((2, T, 1, K, 4), 2.0 ** -20, np.float32)
    run(torch, dev, rng, [1] * T, starts, K, d, 0, rope, k=k, table=table, P=T, pools=pools, scales=scales, gaps=False)
