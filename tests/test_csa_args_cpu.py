"""fm_qk_norm_rope, fm_csa_attn and fm_csa_attn_tree refuse bad arguments on the
host, before they touch a GPU; the Python wrappers check types, shapes and
strides."""
import pytest

FAKE = 4096  # never dereferenced: validation fails first
NOT_THE_DEVICE = "^(?!the tensors are on the CPU)"  # refused for another reason than that


@pytest.fixture(scope="module")
def fm():
    import os
    import sparse_attention_kv_c4_gb300 as fm
    if not os.path.exists(fm.LIB_PATH):
        from sparse_attention_kv_c4_gb300 import _build
        _build.build()
    fm.lib()
    return fm


def test_norm_rope_refusals(fm):
    f = fm.lib().fm_qk_norm_rope
    good = dict(pos=FAKE, T=4, d=512, rope=64, base=160000.0, factor=16.0, orig=65536.0, fast=32.0, slow=1.0, eps=1e-6,
                q=FAKE, qs=64 * 512, nq=64, qg=FAKE, qo=FAKE, k=FAKE, ks=512, nk=1, kg=FAKE, ko=None, kp=FAKE, P=4,
                kps=64 * 512, kc=FAKE, stream=None)

    def call(**new):
        assert set(new) <= set(good)
        return f(*dict(good, **new).values())
    for bad in (dict(T=-1), dict(nq=-1), dict(nq=4096), dict(d=0), dict(d=12), dict(d=1032), dict(rope=-2), dict(rope=3),
                dict(rope=258), dict(d=32, rope=34), dict(base=1.0), dict(factor=0.5), dict(orig=0.0), dict(fast=1.0),
                dict(base=float("nan")),
                dict(base=float("inf")), dict(factor=float("inf")), dict(orig=float("inf")), dict(fast=float("inf")),
                dict(slow=float("-inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(q=None),
                dict(qo=None), dict(k=None), dict(kp=None), dict(kc=None), dict(P=-1), dict(P=(1 << 25) + 1),
                dict(kps=64 * 512 - 8), dict(kps=64 * 512 + 4), dict(qs=64 * 512 - 8), dict(qs=64 * 512 + 4),
                dict(ks=504), dict(ks=513), dict(pos=FAKE + 4), dict(q=FAKE + 8), dict(qo=FAKE + 2), dict(qg=FAKE + 2),
                dict(k=FAKE + 2), dict(kg=FAKE + 8), dict(ko=FAKE + 8), dict(kp=FAKE + 8), dict(kc=FAKE + 2)):
        assert call(**bad) == 1, bad
        assert "fm_qk_norm_rope" in fm.fm_last_error()
    assert call(T=0, q=None, k=None, pos=None) == 0
    assert call(nq=0, nk=0) == 0


def test_attention_refusals(fm):
    f, ft = fm.lib().fm_csa_attn, fm.lib().fm_csa_attn_tree
    page = 64 * 512
    good = dict(q=FAKE, T=4, H=64, d=512, kv=FAKE, P=9, kvs=page, pt=FAKE, B=4, R=3, seq=FAKE, pos=FAKE, window=128,
                n_sink=4, cp=FAKE, Pc=9, cps=page, cells=FAKE, k=512, sink=FAKE, scale=0.04)
    tail = dict(out=FAKE, lse=FAKE, ws=None, wsb=0, stream=None)
    tree = dict(mask=FAKE, words=1, base=FAKE)

    def call(**new):
        assert set(new) <= set(good) | set(tail)
        a = dict(good, **{k: v for k, v in new.items() if k in good})
        z = dict(tail, **{k: v for k, v in new.items() if k in tail})
        first = f(*a.values(), *z.values())
        assert ft(*a.values(), *tree.values(), *z.values()) == first  # both entry points refuse alike
        return first
    for bad in (dict(d=128), dict(T=-1), dict(H=0), dict(H=1025), dict(T=1 << 23, H=2), dict(T=1 << 22, H=65), dict(B=-1), dict(R=-1),
                dict(R=(1 << 19) + 1), dict(window=-1), dict(n_sink=-1), dict(k=-1), dict(k=1025), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(P=-1), dict(kv=None),
                dict(kv=FAKE + 8), dict(kvs=page - 512), dict(kvs=page + 8), dict(P=1 << 25), dict(kvs=1 << 45),
                dict(Pc=-1), dict(cp=None), dict(cps=page + 64), dict(Pc=1 << 25), dict(seq=None, T=5), dict(q=None),
                dict(pos=None), dict(out=None), dict(cells=None), dict(pt=None), dict(q=FAKE + 8), dict(out=FAKE + 2),
                dict(pos=FAKE + 4), dict(pt=FAKE + 2), dict(seq=FAKE + 1), dict(cells=FAKE + 2), dict(sink=FAKE + 2),
                dict(lse=FAKE + 2)):
        assert call(**bad) == 1, bad
        assert "fm_csa_attn" in fm.fm_last_error()
    assert call(T=0) == 0
    for bad in (dict(mask=None), dict(words=0), dict(words=33), dict(base=None), dict(mask=FAKE + 2), dict(base=FAKE + 4)):
        assert ft(*good.values(), *dict(tree, **bad).values(), *tail.values()) == 1, bad
    need = fm.fm_csa_attn_workspace(4, 64)
    if need:
        assert call() == 5 and call(ws=256, wsb=need - 1) == 5 and call(ws=128, wsb=need) == 5
    assert fm.fm_csa_attn_workspace(-1, 64) == 0 and fm.fm_csa_attn_workspace(4, 0) == 0


def test_python_wrappers_check_their_tensors(fm):
    import torch
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(q=bf(2, 4, 512), kv_pool=bf(3, 64, 512), page_table=i32(2, 2), pos=torch.zeros(2, dtype=torch.int64),
                out=bf(2, 4, 512), window=8)
    for bad in (dict(q=bf(2, 4, 512).float()), dict(q=bf(4, 2, 512).transpose(0, 1)), dict(kv_pool=bf(3, 32, 512)),
                dict(kv_pool=bf(3, 64, 1024)[..., ::2]), dict(page_table=i32(2, 2).long()), dict(pos=i32(2)),
                dict(pos=torch.zeros(3, dtype=torch.int64)), dict(out=bf(2, 4, 256)), dict(seq=i32(3)),
                dict(cells=i32(2, 5)), dict(cell_pool=bf(3, 64, 512)), dict(cell_pool=bf(3, 64, 512), cells=i32(3, 5)),
                dict(cell_pool=bf(3, 64, 512), cells=i32(5, 2).t()), dict(sink_logit=torch.zeros(3)),
                dict(lse_out=torch.zeros(2, 5)), dict(workspace=i32(64))):
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_csa_attn(**dict(good, **bad), stream=0)
    for bad in (dict(tree_mask=i32(3, 1)), dict(tree_base=i32(2)), dict(tree_mask=torch.zeros(2, 1))):
        args = dict(good, tree_mask=i32(2, 1), tree_base=torch.zeros(2, dtype=torch.int64))
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_csa_attn_tree(**dict(args, **bad), stream=0)
    pos = torch.zeros(2, dtype=torch.int64)
    for bad in (dict(), dict(q=bf(2, 4, 64)), dict(q=bf(2, 4, 64), q_out=bf(2, 4, 32)), dict(k=bf(2, 1, 64)),
                dict(k=bf(2, 1, 64), k_pool=bf(2, 64, 64)), dict(k=bf(2, 1, 64), k_pool=bf(2, 32, 64), k_cell=i32(2)),
                dict(q=bf(2, 64, 4).transpose(1, 2), q_out=bf(2, 4, 64)),
                dict(q=bf(2, 4, 64), q_out=bf(2, 4, 64), q_gain=bf(32))):
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_qk_norm_rope(pos, **bad, stream=0)
    with pytest.raises(TypeError):
        fm.fm_qk_norm_rope(pos, q=bf(2, 4, 64), q_out=bf(2, 4, 64), rope_size=3)


def test_python_wrappers_refuse_tensors_of_the_cpu(fm):
    import torch
    q, pos = torch.zeros((2, 4, 512), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    args = dict(q=q, kv_pool=torch.zeros((3, 64, 512), dtype=torch.bfloat16), pos=pos, out=q.clone(), window=8,
                page_table=torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="on the CPU"):
        fm.fm_csa_attn(**args, stream=0)
    with pytest.raises(ValueError, match="on the CPU"):
        fm.fm_csa_attn_tree(**args, tree_mask=torch.zeros((2, 1), dtype=torch.int32), tree_base=pos, stream=0)
    with pytest.raises(ValueError, match="on the CPU"):
        fm.fm_qk_norm_rope(pos, q=q, q_out=q.clone(), stream=0)


def test_packed_arguments_are_the_same_call(fm):
    """The struct forms refuse what the calls refuse, with the same words: every
    field is where the struct's reader expects it."""
    L, page = fm.lib(), 64 * 512
    words = lambda call, args: (call(*args), fm.fm_last_error())
    none = lambda args: [0 if a is None else a for a in args]
    good = [FAKE, 4, 512, 64, 160000.0, 16.0, 65536.0, 32.0, 1.0, 1e-6, FAKE, page, 64, FAKE, FAKE, FAKE, 512, 1, FAKE,
            FAKE, FAKE, 4, page, FAKE, None]
    for at, bad in ((0, None), (0, FAKE + 4), (1, -7), (2, 12), (3, 3), (4, 1.0), (5, 0.5), (6, 0.0), (7, 1.0), (8, 32.0),
                    (9, -1.0), (10, None), (11, 8), (12, -5), (13, FAKE + 2), (14, None), (15, FAKE + 2), (16, 504),
                    (17, 4095), (18, FAKE + 8), (19, FAKE + 8), (20, FAKE + 8), (21, -1), (22, page + 4), (23, None)):
        args = good[:at] + [bad] + good[at + 1:]
        want = words(L.fm_qk_norm_rope, args)
        assert want[0] == 1 and words(L.fm_qk_norm_rope_packed, [fm._QK_ARGS.pack(*none(args))]) == want, (at, bad)
    head = [FAKE, 4, 64, 512, FAKE, 9, page, FAKE, 4, 3, FAKE, FAKE, 128, 4, FAKE, 9, page, FAKE, 512, FAKE, 0.04]
    tree, tail = [FAKE, 1, FAKE], [FAKE, FAKE, 256, 8, None]
    flat = head + tree + tail
    for at, bad in ((0, None), (1, -1), (2, 2000), (3, 128), (4, FAKE + 8), (5, -1), (6, page + 8), (7, FAKE + 2), (8, -2),
                    (9, 1 << 20), (10, FAKE + 1), (11, None), (12, -9), (13, -3), (14, None), (15, -1), (16, 64), (17, None),
                    (18, 1025), (19, FAKE + 2), (20, -2.0), (21, None), (22, 33), (23, FAKE + 4), (24, None), (25, FAKE + 2),
                    (26, 128), (27, 9)):
        args = flat[:at] + [bad] + flat[at + 1:]
        want = words(L.fm_csa_attn_tree, args)
        assert want[0] in (1, 5)
        pack = fm._ATTN_ARGS.pack
        assert words(L.fm_csa_attn_packed, [pack(*none(args[:21] + [1] + args[21:]))]) == want, (at, bad)
        if not 21 <= at <= 23:
            want = words(L.fm_csa_attn, args[:21] + args[24:])
            assert words(L.fm_csa_attn_packed, [pack(*none(args[:21] + [0] + args[21:]))]) == want, (at, bad)
    assert L.fm_qk_norm_rope_packed(None) == 1 and L.fm_csa_attn_packed(None) == 1
