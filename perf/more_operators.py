"""The operators of a dense layer of grouped heads and the cases they are measured on.

  prompt  fm_prompt_attn     causal attention over packed prompts
  append  fm_kv_append_fp8   keys and values into the paged 8-bit cache, rotation on the way, the step's queries turned too
  attn    fm_kv_attn_fp8     attention over that cache: decode, and a few drafted tokens a sequence

``run`` computes the plain form in elementary torch operations, or, where ``own`` is set, makes the calls that a
user of the package makes.
"""
import math

import torch

own = False

PAGE = 64    # tokens in a cache page
BLOCK = 16   # tokens that share a scale
TOP = 448.0  # E4M3's largest value
ROPE = dict(rope_base=160000.0, rope_factor=16.0, rope_orig_len=65536.0, rope_beta_fast=32.0, rope_beta_slow=1.0)


def listed():
    return [
        # one request's next token of a long context: latency only
        dict(name="append_decode_1", op="append", B=1, n=1, pos=1048575, H=32, K=8, d=128, rope=64, ragged=False),
        # the decode batch of the 256K context (76 requests), requests of every length
        dict(name="append_decode_76", op="append", B=76, n=1, pos=262143, H=64, K=8, d=128, rope=64, ragged=True),
        # prompts of odd lengths, behind a cached prefix that ends inside a block
        dict(name="append_prompts_5", op="append", B=5, n=613, pos=649, H=20, K=4, d=96, rope=64, ragged=True),
        # a prefill step of 4096 tokens at position 262147
        dict(name="append_prefill_4096", op="append", B=1, n=4096, pos=266242, H=64, K=8, d=128, rope=64, ragged=False),
        # a short chat's next token: 37 tokens of history
        dict(name="attn_first_1", op="attn", B=1, n=1, pos=36, H=32, K=8, d=128, window=None, sink=False, ragged=False),
        # a decode batch of 30 requests of every length up to 32K
        dict(name="attn_decode_30", op="attn", B=30, n=1, pos=32767, H=64, K=8, d=128, window=None, sink=True, ragged=True),
        # one request's next token at 1M tokens: the cache is streamed once
        dict(name="attn_long_1", op="attn", B=1, n=1, pos=1048575, H=32, K=4, d=128, window=None, sink=False, ragged=False),
        # five drafted tokens behind each of eight requests, a sliding window of odd length, five heads a group
        dict(name="attn_drafts_8", op="attn", B=8, n=5, pos=16383, H=40, K=8, d=64, window=8191, sink=True, ragged=True),
        # a short chat's first turn
        dict(name="prompt_first_37", op="prompt", B=1, n=37, past=0, H=32, K=8, d=128, window=None, sink=False, ragged=False),
        # prompts of odd lengths, 20 heads, a cached prefix before each
        dict(name="prompt_5", op="prompt", B=5, n=613, past=131, H=20, K=4, d=96, window=None, sink=True, ragged=True),
        # layers with a sliding window over packed prompts of up to 4096 tokens
        dict(name="prompt_window_4", op="prompt", B=4, n=4096, past=0, H=32, K=8, d=64, window=1021, sink=True, ragged=True),
        # a prompt of 8192 tokens
        dict(name="prompt_8192", op="prompt", B=1, n=8192, past=0, H=32, K=8, d=128, window=None, sink=False, ragged=False),
    ]


MOST_PAIRS = 8192 * 8192 * 32       # query x key x head products that a prompt's plain form holds
MOST_CACHE = 1048576 * 4 * 128      # elements of keys in the largest listed cache
MOST_ROWS = 4096 * (64 + 16) * 128  # elements that the largest listed append moves


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "prompt"])
    d, K = rng.choice([64, 128, 128, 16 * rng.randint(1, 8)]), rng.choice([1, 2, 4, 8, 8, 16, rng.randint(1, 16)])
    H = K * rng.choice([1, 2, 4, 4, 8, rng.randint(1, 16)])
    while H > 128:
        H -= K
    B, window = _spread(rng, 1, 96), rng.choice([None, None, _spread(rng, 1, 16384)])
    case = dict(op=op, H=H, K=K, d=d, ragged=rng.random() < 0.6)
    if op == "append":
        n = rng.choice([1, _spread(rng, 1, 4096)])
        while B * n > 1 and B * n * (H + 2 * K) * d > MOST_ROWS:
            B, n = max(1, B // 2), max(1, n // 2)
        return dict(case, B=B, n=n, pos=n - 1 + _spread(rng, 1, 1 << 18), rope=2 * rng.randint(0, d // 2))
    case.update(window=window, sink=rng.random() < 0.5)
    if op == "attn":
        n, length = rng.choice([1, 1, rng.randint(1, 8)]), _spread(rng, 1, 1 << 19)
        while length * B > 1 and (length + n) * B * K * d > MOST_CACHE:
            B, length = max(1, B // 2), max(1, length // 2)
        return dict(case, B=B, n=n, pos=n - 1 + length)
    n, past = _spread(rng, 1, 8192), rng.choice([0, 0, _spread(rng, 1, 4096)])
    while B * n > 1 and B * n * (n + past) * H > MOST_PAIRS:
        B, n = max(1, B // 2), max(1, n // 2)
    while past and B * n * (n + past) * H > MOST_PAIRS:
        past //= 2
    return dict(case, B=B, n=n, past=past)


# ------------------------------------------------------------------------------------------------ inputs


def _sequences(case):
    """(new tokens, tokens before them) of each sequence."""
    B, n = case["B"], case["n"]
    out = []
    for b in range(B):
        nb = max(1, n - (13 * b) % n) if case["ragged"] else n
        if case["op"] == "prompt":
            out.append((nb, case["past"] * (B - b) // B if case["ragged"] else case["past"]))
        else:
            last = case["pos"] * (b + 1) // B if case["ragged"] else case["pos"]
            out.append((nb, max(0, last + 1 - nb)))
    return out


def _offsets(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _paged(case, cpu):
    """Pages in a random order: those that the new tokens and what they see are on; -1 elsewhere."""
    held = []
    for n, past in _sequences(case):
        low = past // BLOCK * BLOCK if case["op"] == "append" else 0 if case["window"] is None else max(0, past + 1 - case["window"])
        held.append((low // PAGE, (past + n - 1) // PAGE + 1))
    pages = sum(e - s for s, e in held) + 3
    order = torch.randperm(pages, generator=cpu).to(torch.int32)
    table, at = torch.full((len(held), max(e for _, e in held)), -1, dtype=torch.int32), 0
    for b, (s, e) in enumerate(held):
        table[b, s:e] = order[at:at + e - s]
        at += e - s
    return table.cuda(), pages


def _cells(shape, g):
    """A pool [P, K, 64, d] of codes and its scales [P, K, 64 / BLOCK]: normal values, each block and head of its own size."""
    P, K, _, d = shape
    x = torch.randn((P, K, PAGE // BLOCK, BLOCK * d), generator=g, device="cuda")
    size = (0.3 * torch.randn((P, K, PAGE // BLOCK), generator=g, device="cuda")).exp()
    scale = _need(x.abs().amax(-1) * size)
    x.mul_((size / scale)[..., None])
    return x.to(torch.float8_e4m3fn).view(P, K, PAGE, d).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    seqs, H, K, d = _sequences(case), case["H"], case["K"], case["d"]
    T = sum(n for n, _ in seqs)
    s = dict(case=case, cu=_offsets([n for n, _ in seqs]))
    if case["op"] == "prompt":
        keys = sum(n + past for n, past in seqs)
        s.update(q=new(T, H, d), k=new(keys, K, d), v=new(keys, K, d), cu_k=_offsets([n + past for n, past in seqs]))
    else:
        s["table"], pages = _paged(case, cpu)
        s["start"] = torch.tensor([past for _, past in seqs], dtype=torch.int64).cuda()
        for x in ("k", "v"):
            s[x + "_pool"], s[x + "_scale"] = _cells((pages, K, PAGE, d), g)
        s["q"] = new(T, H, d)
    if case["op"] == "append":  # the projections' output: a token's query heads, its key heads, its value heads
        fused = 2 * new(T, (H + 2 * K) * d)
        s["q"], s["q_out"] = fused[:, :H * d].view(T, H, d), torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
        s["k"], s["v"] = fused[:, H * d:(H + K) * d].view(T, K, d), fused[:, (H + K) * d:].view(T, K, d)
    else:
        s["sink"] = torch.randn(H, generator=g, device="cuda") if case["sink"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        s["most"] = max(n + past for n, past in seqs)
    return s


# ------------------------------------------------------------------------------------------------ plain form


def _need(amax):
    """The least power of two, from 2^-100 on, that brings amax to at most TOP."""
    m, e = torch.frexp(amax / TOP)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e + 127) << 23).view(torch.float32)


def _tokens(s):
    """The sequence and the place in it of each new token."""
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device="cuda"), cu.diff(), output_size=s["q"].shape[0])
    return seq, torch.arange(s["q"].shape[0], device="cuda") - cu[seq]


def _turned(x, angle, rope):
    x = x.double()
    flat, a, b = x[..., :x.shape[-1] - rope], x[..., x.shape[-1] - rope::2], x[..., x.shape[-1] - rope + 1::2]
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]
    return torch.cat([flat, torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)], -1)


def _append_plain(s):
    rope = s["case"]["rope"]
    seq, i = _tokens(s)
    start = s["start"][seq]
    pos = start + i
    theta = ROPE["rope_base"] ** (-torch.arange(0, rope, 2, dtype=torch.float64, device="cuda") / max(rope, 1))
    turns = ROPE["rope_orig_len"] * theta / (2 * math.pi)
    keep = ((turns - ROPE["rope_beta_slow"]) / (ROPE["rope_beta_fast"] - ROPE["rope_beta_slow"])).clamp(0, 1)
    angle = pos.double()[:, None] * (theta * (keep + (1 - keep) / ROPE["rope_factor"]))
    s["q_out"].copy_(_turned(s["q"], angle, rope))
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    # the cells of a sequence's first block that were there before this call
    lead = s["start"] // BLOCK * BLOCK + torch.arange(BLOCK, device="cuda")[:, None]
    old = (lead < s["start"]).T
    old_page = s["table"].gather(1, (lead.T // PAGE)).long()[old]
    old_slot = (lead.T % PAGE)[old]
    began = pos // BLOCK * BLOCK >= start
    for name, x in (("k", _turned(s["k"], angle, rope)), ("v", s["v"].double())):
        pool, scale = s[name + "_pool"].view(torch.float8_e4m3fn), s[name + "_scale"]
        amax = torch.zeros(scale.shape, dtype=torch.float64, device="cuda").transpose(1, 2).contiguous()
        flat = amax.view(-1, x.shape[1])
        at = (page * (PAGE // BLOCK) + slot // BLOCK)[:, None].expand(-1, x.shape[1])
        flat.scatter_reduce_(0, at, x.abs().amax(-1), "amax")
        before = scale[page, :, slot // BLOCK]
        now = _need(flat.gather(0, at))
        now = torch.where(began[:, None], now, torch.maximum(now, before))
        kept, kept_before = pool.view(torch.uint8)[old_page, :, old_slot].view(torch.float8_e4m3fn), scale[old_page, :, old_slot // BLOCK]
        scale[page, :, slot // BLOCK] = now
        ratio = kept_before / scale[old_page, :, old_slot // BLOCK]
        pool.view(torch.uint8)[old_page, :, old_slot] = (kept.float() * ratio[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        pool.view(torch.uint8)[page, :, slot] = (x / now[..., None].double()).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return _append_outputs(s)


def _append_outputs(s):
    return {"q": s["q_out"], "k": s["k_pool"].view(torch.float8_e4m3fn), "v": s["v_pool"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attend(s, q, keys, values, seen):
    """q [B, n, H, d], keys and values [B, m, K, d] in fp32, seen [B, n, m] -> out [B, n, H, d], lse [B, n, H]."""
    B, n, H, d = q.shape
    K, m = keys.shape[2], keys.shape[1]
    rows = q.view(B, n, K, H // K, d).permute(0, 2, 1, 3, 4).reshape(B, K, n * (H // K), d)
    score = torch.matmul(rows, keys.permute(0, 2, 3, 1)).mul_(d ** -0.5).view(B, K, n, H // K, m)
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    below = total if s["sink"] is None else total + (s["sink"].view(K, 1, H // K, 1) - top).exp()
    out = torch.matmul(weight.view(B, K, -1, m), values.transpose(1, 2)).view(B, K, n, H // K, d) / below.clamp(min=1e-38)
    return out.permute(0, 2, 1, 3, 4).reshape(B, n, H, d), (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B, n, H)


def _attention_plain(s):
    case = s["case"]
    seq, i = _tokens(s)
    cu = s["cu"].long()
    lane = torch.arange(case["n"], device="cuda")
    q = s["q"][(cu[:-1, None] + lane).clamp(max=s["q"].shape[0] - 1)].float()  # rows past a sequence's end go nowhere
    if case["op"] == "prompt":
        last = s["cu_k"].long().diff() - 1
        past = last + 1 - cu.diff()
        at = torch.arange(s["most"], device="cuda").expand(case["B"], -1)
        rows = (s["cu_k"].long()[:-1, None] + at).clamp(max=s["k"].shape[0] - 1)
        keys, values = s["k"][rows].float(), s["v"][rows].float()
    else:
        past = s["start"]
        last = past + cu.diff() - 1
        width = s["most"] if case["window"] is None else min(s["most"], case["window"] + case["n"] - 1)
        at = (last - width + 1).clamp(min=0)[:, None] + torch.arange(width, device="cuda")
        page = s["table"].gather(1, (at // PAGE).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
        keys, values = (s[x + "_pool"].view(torch.float8_e4m3fn).view(torch.uint8)[page, :, at % PAGE].view(torch.float8_e4m3fn).float()
                        * s[x + "_scale"][page, :, at % PAGE // BLOCK][..., None] for x in ("k", "v"))
    pos = past[:, None] + lane
    seen = (at[:, None, :] <= pos[:, :, None]) & (at <= last[:, None])[:, None, :]
    if case["window"] is not None:
        seen &= at[:, None, :] > pos[:, :, None] - case["window"]
    out, lse = _attend(s, q, keys, values, seen)
    s["out"].copy_(out[seq, i])
    s["lse"].copy_(lse[seq, i])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    if not own:
        return _append_plain(s) if case["op"] == "append" else _attention_plain(s)
    import sparse_attention_kv_c4_gb300 as fm
    if case["op"] == "append":
        fm.fm_kv_append_fp8(s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["start"],
                            cu_tokens=s["cu"], q=s["q"], q_out=s["q_out"], rope_dim=case["rope"], **ROPE)
        return _append_outputs(s)
    if case["op"] == "prompt":
        fm.fm_prompt_attn(s["q"], s["k"], s["v"], s["out"], cu_q=s["cu"], cu_k=s["cu_k"], window=case["window"],
                          sink_logit=s["sink"], lse_out=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if "workspace" not in s:  # a user's program keeps it
        size = fm.fm_kv_attn_fp8_workspace(s["q"].shape[0], case["H"], case["K"], case["d"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    fm.fm_kv_attn_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["start"], s["out"],
                      cu_tokens=s["cu"], window=case["window"], sink_logit=s["sink"], lse_out=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------ work, exact values


def work(case):
    seqs, H, K, d = _sequences(case), case["H"], case["K"], case["d"]
    T = sum(n for n, _ in seqs)
    if case["op"] == "append":
        blocks = sum((past + n - 1) // BLOCK - past // BLOCK + 1 for n, past in seqs)
        return {"bytes": T * d * (4 * H + 6 * K) + 8 * blocks * K, "flops": 3 * T * (H + K) * case["rope"]}
    window = case["window"] or 1 << 60
    pairs = read = 0
    for n, past in seqs:
        full = max(0, min(n, past + n - window))  # tokens whose window is full
        pairs += full * window + (n - full) * (past + 1) + (n - full) * (n - full - 1) // 2 if full < n else n * window
        read += min(past + n, window + n - 1)
    cell = 4 * K * d if case["op"] == "prompt" else 2 * K * d + 8 * K // BLOCK
    return {"bytes": 4 * T * H * d + 4 * T * H + read * cell, "flops": 4 * d * H * pairs}


def _e4m3(x):
    """Values in 64 bits rounded to E4M3's, ties to even."""
    exponent = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1]
    step = ((exponent.long() + 1019) << 52).view(torch.float64)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _exact_append(case, s):
    rope, out = case["rope"], {}
    freq = []
    for i in range(rope // 2):
        theta = ROPE["rope_base"] ** (-2.0 * i / rope)
        ramp = (ROPE["rope_orig_len"] * theta / (2 * math.pi) - ROPE["rope_beta_slow"]) / (ROPE["rope_beta_fast"] - ROPE["rope_beta_slow"])
        ramp = min(1.0, max(0.0, ramp))
        freq.append((1 - ramp) * theta / ROPE["rope_factor"] + ramp * theta)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")

    def turn(x, pos):
        x = x.double().clone()
        if rope:
            pair = torch.view_as_complex(x[..., x.shape[-1] - rope:].unflatten(-1, (-1, 2)).contiguous())
            unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * freq)
            x[..., x.shape[-1] - rope:] = torch.view_as_real(pair * unit[:, None, :]).flatten(-2)
        return x
    out["q"] = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    pools = {x: (s[x + "_pool"].view(torch.float8_e4m3fn).double(), s[x + "_scale"].double()) for x in ("k", "v")}
    table, t = s["table"].tolist(), 0
    for b, (n, past) in enumerate(_sequences(case)):
        pos = past + torch.arange(n, device="cuda")
        out["q"][t:t + n] = turn(s["q"][t:t + n], pos)
        rows = {"k": turn(s["k"][t:t + n], pos), "v": s["v"][t:t + n].double()}
        for j in range(past // BLOCK, (past + n - 1) // BLOCK + 1):
            page, first = table[b][j * BLOCK // PAGE], j * BLOCK % PAGE
            lo, hi = max(past, j * BLOCK), min(past + n, (j + 1) * BLOCK)
            for x, (pool, scale) in pools.items():
                new = rows[x][lo - past:hi - past].transpose(0, 1)
                top = new.abs().amax((1, 2))
                s_new = torch.tensor([2.0 ** e for e in range(-100, 128)], dtype=torch.float64, device="cuda")
                s_new = s_new[(TOP * s_new[None, :] < top[:, None]).sum(-1)]
                if lo > j * BLOCK:
                    s_old = scale[page, :, first // BLOCK].clone()
                    s_new = torch.maximum(s_new, s_old)
                    kept = pool[page, :, first:first + lo - j * BLOCK]
                    kept.copy_(_e4m3(kept * (s_old / s_new)[:, None, None]))
                scale[page, :, first // BLOCK] = s_new
                pool[page, :, first + lo - j * BLOCK:first + hi - j * BLOCK] = _e4m3(new / s_new[:, None, None])
        t += n
    for x, (pool, scale) in pools.items():
        out[x], out[x + "_scale"] = pool, scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    H, K, d = case["H"], case["K"], case["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    t = u = 0
    for b, (n, past) in enumerate(_sequences(case)):
        low = 0 if case["window"] is None else max(0, past + 1 - case["window"])
        at = torch.arange(low, past + n, device="cuda")
        if case["op"] != "prompt":
            pages = s["table"][b][at // PAGE].long()
        for g in range(K):
            if case["op"] == "prompt":
                keys, values = (s[x][u + low:u + past + n, g].double() for x in ("k", "v"))
            else:
                keys, values = (s[x + "_pool"].view(torch.float8_e4m3fn)[:, g].double()[pages, at % PAGE]
                                * s[x + "_scale"][:, g].double()[pages, at % PAGE // BLOCK][:, None] for x in ("k", "v"))
            pos = past + torch.arange(n, device="cuda")
            seen = at[None, :] <= pos[:, None]
            if case["window"] is not None:
                seen &= at[None, :] > pos[:, None] - case["window"]
            for h in range(g * (H // K), (g + 1) * (H // K)):
                x = (s["q"][t:t + n, h].double() @ keys.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[t:t + n, h] = z
                z = z if s["sink"] is None else torch.logaddexp(z, s["sink"][h].double())
                out[t:t + n, h] = torch.where(z[:, None] > -math.inf, (x - z[:, None]).exp(), 0) @ values
        t += n
        u += n + past
    return {"out": out, "lse": lse}
