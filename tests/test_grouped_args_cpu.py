"""fm_prompt_attn, fm_kv_append_fp8 and fm_kv_attn_fp8 refuse bad arguments on the host, before
they touch a GPU; the Python wrappers check types, shapes and strides."""
import numpy as np
import pytest

import grouped_ref as gr

FAKE = 4096  # never dereferenced: validation fails first
NOT_THE_DEVICE = "^(?!the tensors are on the CPU)"


@pytest.fixture(scope="module")
def fm():
    import os
    import sparse_attention_kv_c4_gb300 as fm
    if not os.path.exists(fm.LIB_PATH):
        from sparse_attention_kv_c4_gb300 import _build
        _build.build()
    fm.lib()
    return fm


NAN, INF = float("nan"), float("inf")
APPEND = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, T=4, n_k=8, d=128, n_h=32, q=FAKE, qs=4096, qo=FAKE, kp=FAKE, vp=FAKE, ksc=FAKE,
              vsc=FAKE, P=9, page=65536, sst=32, pt=FAKE, B=4, R=3, start=FAKE, cu=FAKE, base=160000.0, factor=16.0,
              orig=65536.0, fast=32.0, slow=1.0, rope=64, stream=0)
KV = dict(q=FAKE, qs=4096, T=4, n_h=32, n_k=8, d=128, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE, P=9, page=65536, sst=32, pt=FAKE, B=4,
          R=3, start=FAKE, cu=FAKE, window=128, sink=FAKE, scale=0.1, out=FAKE, lse=FAKE, ws=0, wsb=0, stream=0)
PROMPT = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, T=4, Tk=6, n_h=32, n_k=8, d=128, B=2, cuq=FAKE, cuk=FAKE, window=9,
              sink=FAKE, scale=0.1, out=FAKE, lse=FAKE, stream=0)
CACHE = (dict(P=-1), dict(P=(1 << 25) + 1), dict(page=65520), dict(page=65544), dict(page=1 << 38), dict(sst=28), dict(sst=34),
         dict(sst=1 << 38), dict(pt=0), dict(pt=FAKE + 2), dict(R=-1), dict(R=(1 << 19) + 1), dict(B=-1), dict(B=(1 << 24) + 1),
         dict(kp=0), dict(vp=0), dict(ksc=0), dict(vsc=0), dict(kp=FAKE + 8), dict(vp=FAKE + 4), dict(ksc=FAKE + 4),
         dict(vsc=FAKE + 8), dict(start=0), dict(start=FAKE + 4), dict(cu=FAKE + 2), dict(cu=0, T=5))
HEADS = (dict(n_h=0), dict(n_h=1025), dict(n_k=0), dict(n_k=3), dict(n_k=-8), dict(d=0), dict(d=8), dict(d=72), dict(d=144),
         dict(n_h=1024, n_k=4), dict(T=-1))
SCORES = (dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(scale=3e38), dict(out=0),
          dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(sink=FAKE + 1), dict(q=0), dict(q=FAKE + 8), dict(qs=4088), dict(qs=4100),
          dict(qs=1 << 39))


@pytest.mark.parametrize("name,pack,good,bads", [
    ("fm_kv_append_fp8", "_APPEND_ARGS", APPEND, CACHE + HEADS + (
        dict(T=1 << 24), dict(k=0), dict(k=FAKE + 8), dict(ks=1016), dict(ks=1028), dict(v=0), dict(v=FAKE + 2), dict(vs=1000),
        dict(vs=1025), dict(q=FAKE + 8), dict(qs=4088), dict(qs=4100), dict(qo=0), dict(qo=FAKE + 4), dict(rope=-2), dict(rope=3),
        dict(rope=130), dict(base=1.0), dict(base=INF), dict(base=NAN), dict(factor=0.5), dict(factor=INF), dict(orig=0.0),
        dict(orig=INF), dict(fast=1.0), dict(fast=INF), dict(slow=-INF))),
    ("fm_kv_attn_fp8", "_KV_ATTN_ARGS", KV, CACHE + HEADS + SCORES + (dict(T=1 << 24),)),
    ("fm_prompt_attn", "_PROMPT_ARGS", PROMPT, HEADS + SCORES + (
        dict(T=1 << 30), dict(Tk=-1), dict(Tk=1 << 30), dict(B=-1), dict(B=(1 << 24) + 1), dict(k=0), dict(v=0), dict(k=FAKE + 8),
        dict(v=FAKE + 8), dict(ks=1016), dict(vs=1020), dict(cuq=0), dict(cuq=0, cuk=0), dict(cuk=0), dict(cuq=FAKE + 2),
        dict(cuk=FAKE + 1))),
])
def test_refusals(fm, name, pack, good, bads):
    call = lambda **new: getattr(fm.lib(), name)(getattr(fm, pack).pack(*dict(good, **new).values()))
    for bad in bads:
        assert set(bad) <= set(good)
        assert call(**bad) == 1, bad
        assert name in fm.fm_last_error()
    assert call(T=0, **({"Tk": 0, "k": 0, "v": 0} if "Tk" in good else {})) == 0
    assert getattr(fm.lib(), name)(None) == 1


def test_workspace(fm):
    size = fm.fm_kv_attn_fp8_workspace
    for bad in ((-1, 32, 8, 128), (4, 0, 8, 128), (4, 32, 7, 128), (4, 32, 8, 120), (4, 1025, 1025, 64)):
        assert size(*bad) == 0
    need = size(4, 32, 8, 128)
    call = lambda **new: fm.lib().fm_kv_attn_fp8(fm._KV_ATTN_ARGS.pack(*dict(KV, **new).values()))
    if need:
        assert call() == 5 and call(ws=256, wsb=need - 1) == 5 and call(ws=128, wsb=need) == 5


def test_python_wrappers_check_their_tensors(fm):
    import torch
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32, i64 = (lambda *s: torch.zeros(s, dtype=torch.int32)), (lambda *s: torch.zeros(s, dtype=torch.int64))
    u8, f32 = (lambda *s: torch.zeros(s, dtype=torch.uint8)), (lambda *s: torch.zeros(s))
    cache = dict(k_pool=u8(5, 2, 64, 32), v_pool=u8(5, 2, 64, 32).view(torch.float8_e4m3fn), k_scale=f32(5, 2, 4), v_scale=f32(5, 2, 4),
                 page_table=i32(3, 2), start=i64(3))
    bad_cache = [dict(k_pool=u8(5, 2, 32, 32)), dict(k_pool=u8(5, 64, 2, 32).transpose(1, 2)), dict(v_pool=u8(5, 2, 64, 48)),
                 dict(v_pool=u8(4, 2, 64, 32)), dict(v_pool=u8(5, 2, 64, 32).to(torch.int8)), dict(v_pool=u8(10, 2, 64, 32)[::2]),
                 dict(k_scale=f32(5, 2, 3)), dict(k_scale=f32(5, 2, 4).double()), dict(v_scale=f32(5, 4, 4)[:, :2]),
                 dict(page_table=i64(3, 2)), dict(page_table=i32(2, 3).t()), dict(start=i32(3)), dict(start=i64(2)),
                 dict(cu_tokens=i32(3)), dict(cu_tokens=i64(4)), dict(page_table=i32(4, 2), start=i64(4))]
    append = dict(cache, k=bf(3, 2, 32), v=bf(3, 2, 32))
    for bad in bad_cache + [dict(k=bf(3, 2, 32).float()), dict(v=bf(3, 1, 32)), dict(v=bf(2, 2, 32)), dict(q=bf(3, 4, 32)),
                            dict(q_out=bf(3, 4, 32)), dict(q=bf(3, 4, 32), q_out=bf(3, 4, 16)), dict(q=bf(3, 4, 16), q_out=bf(3, 4, 16)),
                            dict(k=bf(3, 2, 64)[..., ::2])]:
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_kv_append_fp8(**dict(append, **bad), stream=0)
    attn = dict(cache, q=bf(3, 4, 32), out=bf(3, 4, 32))
    for bad in bad_cache + [dict(q=bf(3, 4, 16)), dict(out=bf(3, 4, 32).float()), dict(out=bf(3, 8, 32)[:, ::2]), dict(sink_logit=f32(3)),
                            dict(lse_out=f32(4, 3)), dict(workspace=i32(9))]:
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_kv_attn_fp8(**dict(attn, **bad), stream=0)
    prompt = dict(q=bf(3, 4, 32), k=bf(3, 2, 32), v=bf(3, 2, 32), out=bf(3, 4, 32))
    for bad in (dict(k=bf(3, 2, 16)), dict(v=bf(4, 2, 32)), dict(v=bf(3, 4, 32)), dict(out=bf(2, 4, 32)), dict(cu_q=i64(2)),
                dict(cu_k=i32(2)), dict(cu_q=i32(3), cu_k=i32(2)), dict(sink_logit=f32(2)), dict(lse_out=f32(3)),
                dict(q=bf(4, 3, 32).transpose(0, 1))):
        with pytest.raises(ValueError, match=NOT_THE_DEVICE):
            fm.fm_prompt_attn(**dict(prompt, **bad), stream=0)
    for call, args in ((fm.fm_kv_append_fp8, append), (fm.fm_kv_attn_fp8, attn), (fm.fm_prompt_attn, prompt)):
        with pytest.raises(ValueError, match="on the CPU"):
            call(**args, stream=0)


def test_reference_codes():
    """The tests' E4M3 rounding: exact on its own values, nearest and even between them."""
    assert (gr.e4m3_codes(gr.VALUES[:127]) == np.arange(127)).all() and gr.VALUES[126] == 448
    mid = (gr.VALUES[:126] + gr.VALUES[1:127]) / 2
    assert (gr.e4m3_codes(mid) == np.arange(126) + np.arange(126) % 2).all()
    assert (gr.e4m3_codes(mid * (1 + 1e-9)) == np.arange(126) + 1).all()
    assert [gr.need_scale(x) for x in (0.0, 448.0, 449.0, 3.5, 1e-40)] == [2.0 ** -100, 1, 2, 2.0 ** -7, 2.0 ** -100]


def test_reference_attention_and_append_agree_with_a_dense_softmax():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 4, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    out, lse, _, _ = gr.attend(q, k, v, 6, 1 << 60, None, 0.25)
    s = np.einsum("nhd,mhd->nhm", q, k[:, [0, 0, 1, 1]]) * 0.25
    s[np.broadcast_to(np.arange(9) > 6 + np.arange(3)[:, None, None], s.shape)] = -np.inf
    w = np.exp(s)
    assert np.allclose(lse, np.log(w.sum(-1))) and np.allclose(out, np.einsum("nhm,mhd->nhd", w / w.sum(-1, keepdims=True), v[:, [0, 0, 1, 1]]))
    pools, scales = [np.zeros((1, 2, 64, 16), np.uint8) for _ in "kv"], [np.ones((1, 2, 4), np.float32) for _ in "kv"]
    gr.append(k, v, pools, scales, np.zeros((1, 1), np.int32), np.array([0]), np.array([0, 9]), 0)
    got = gr.VALUES[pools[1][0, :, :9]] * scales[1][0, :, :1, None]
    assert (np.abs(got - v.transpose(1, 0, 2)) <= 2.0 ** -4 * np.abs(v.transpose(1, 0, 2)) + 1e-3).all()
