"""The operators of a CSA layer's attention and the cases they are measured on.

  qk    fm_qk_norm_rope    RMSNorm of each query and key head and the YaRN rotation, keys into their cache cells
  attn  fm_csa_attn        one softmax over the selected chunk cells, the first tokens and the sliding window
  tree  fm_csa_attn_tree   the same for a tree of drafted tokens behind a committed cache

``run`` computes the plain form in elementary torch operations, or, where ``own`` is set, makes the calls that a
user of the package makes.
"""
import math

import torch

own = False

PAGE = 64      # tokens (or chunk cells) in a page
WIDTH = 512    # elements of a cell: the latent that is key and value at once
ROPE = dict(rope_base=160000.0, rope_factor=16.0, rope_orig_len=65536.0, rope_beta_fast=32.0, rope_beta_slow=1.0)
EPS = 1e-6
RATIO = 4      # tokens in a chunk


def listed():
    attn = dict(op="attn", ragged=False, sink=True)
    tree = dict(op="tree", ragged=True, sink=True)
    return [
        # one request's next token: the smallest call, latency only
        dict(name="qk_decode_1", op="qk", T=1, H=64, K=1, d=512, rope=64, pos=1048575),
        # the decode batch of the 256K context (76 requests)
        dict(name="qk_decode_76", op="qk", T=76, H=64, K=1, d=512, rope=64, pos=262143),
        # an odd prompt with grouped heads of the indexer's width
        dict(name="qk_grouped_1021", op="qk", T=1021, H=32, K=8, d=128, rope=64, pos=8191),
        # a prefill step of 4096 tokens
        dict(name="qk_prefill_4096", op="qk", T=4096, H=64, K=1, d=512, rope=64, pos=266239),
        # a short chat's next token: 37 tokens of history, nothing selected yet
        dict(name="attn_first_1", **attn, B=1, n=1, H=64, pos=36, k=0, rows=64, window=128, first=0),
        # the decode batch of the 1M context: 30 requests, top-512 cells, 128-token window, 4 first tokens
        dict(name="attn_decode_30", **attn, B=30, n=1, H=64, pos=1048575, k=512, rows=262144, window=128, first=4),
        # the decode batch of the 256K context with 128 heads and requests of every length up to it
        dict(name="attn_decode_76", op="attn", ragged=True, sink=True, B=76, n=1, H=128, pos=262143, k=512, rows=131072,
             window=128, first=4),
        # decode with a long window of plain tokens and no selection: the cache is streamed once
        dict(name="attn_window_32k", **attn, B=8, n=1, H=64, pos=131071, k=0, rows=64, window=32768, first=64),
        # prompts of odd lengths from their first token on: short windows, few chunks, 20 heads
        dict(name="attn_prompts_5", op="attn", ragged=True, sink=False, B=5, n=613, H=20, pos=612, k=512, rows=4096,
             window=128, first=4),
        # a prefill step of 4096 tokens at position 262144 with top-512 cells
        dict(name="attn_prefill_4096", **attn, B=1, n=4096, H=64, pos=266239, k=512, rows=65536, window=128, first=4),
        # 16 drafted tokens behind each of four requests of a 512K context
        dict(name="tree_4x16", **tree, B=4, n=16, H=64, pos=524287, k=512, rows=131072, window=128, first=4),
        # wide trees of 61 drafted tokens over a 4096-token window
        dict(name="tree_2x61", **tree, B=2, n=61, H=64, pos=32767, k=0, rows=64, window=4096, first=4),
    ]


MOST_KEYS = 4096 * 64 * 644      # token x head x key products of the largest listed attention case
MOST_READ = 4096 * 644           # token x key products of that case: what the plain form gathers
MOST_ELEMENTS = 4096 * 65 * 512  # elements of the largest listed norm


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "attn", "attn", "tree"])
    if op == "qk":
        d = rng.choice([64, 96, 128, 192, 256, 320, 512, 576])
        H, K = rng.randint(1, 128), rng.choice([1, 1, 2, 4, 8])
        T = min(_spread(rng, 1, 8192), max(1, MOST_ELEMENTS // (d * (H + K))))
        return dict(op=op, T=T, H=H, K=K, d=d, rope=min(d, rng.choice([32, 64, 64, 128])),
                    pos=max(T - 1, _spread(rng, 1, 1 << 20)))
    H = rng.choice([rng.randint(1, 128), 64, 64, 128])
    k = rng.choice([0, 512, rng.randint(1, 1024)])
    window, first = _spread(rng, 1, 16384), rng.choice([0, 4, rng.randint(1, 200)])
    B = _spread(rng, 1, 96)
    n = _spread(rng, 1, 1024) if op == "attn" else _spread(rng, 1, 96)
    most = min(MOST_KEYS // H, MOST_READ)
    while B * n > 1 and (B * n > 8192 or B * n * (k + window + first) > most):
        B, n = max(1, B // 2), max(1, n // 2)
    return dict(op=op, B=B, n=n, H=H, pos=max(n - 1, _spread(rng, 1, 1 << 20)), k=k, rows=max(1024, _spread(rng, 1024, 65536)),
                window=window, first=first, ragged=rng.random() < 0.6, sink=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ inputs


def _sequences(case):
    """(new tokens, position of the last one) of each sequence; of a tree, (drafted tokens, last committed position)."""
    B, n, last = case["B"], case["n"], case["pos"]
    if not case["ragged"]:
        return [(n, last)] * B
    out = []
    for b in range(B):
        nb = max(1, n - (13 * b) % n)
        out.append((nb, max(nb - 1, last * (b + 1) // B)))
    return out


def _held(case):
    """The pages of each sequence that its cache still holds: those of the first tokens, the windows and the drafts."""
    pages = []
    for n, last in _sequences(case):
        tree = case["op"] == "tree"
        low = max(0, last + 1 - case["window"] if tree else last - n + 2 - case["window"])
        high = last + n if tree else last
        held = set(range(low // PAGE, high // PAGE + 1))
        first = min(case["first"], last + 1)
        held |= set(range(0, (first + PAGE - 1) // PAGE))
        pages.append(sorted(held))
    return pages


def _attention_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    seqs, held = _sequences(case), _held(case)
    tree = case["op"] == "tree"
    seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, (n, _) in enumerate(seqs)])
    T = seq.numel()
    pages = sum(map(len, held)) + 3
    order = torch.randperm(pages, generator=cpu, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(seqs), max(p[-1] for p in held) + 1), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(held):
        table[b, torch.tensor(p)] = order[at:at + len(p)]
        at += len(p)
    s = dict(q=new(T, case["H"], WIDTH), kv_pool=new(pages, PAGE, WIDTH), page_table=table.cuda(), seq=seq.cuda(),
             sink_logit=torch.randn(case["H"], generator=g, device="cuda") if case["sink"] else None)
    if tree:  # random trees: node i hangs on one of the few before it, or on the last committed token
        words = (max(n for n, _ in seqs) + 31) // 32
        bits = torch.zeros((T, words * 32), dtype=torch.int64)
        pos, t = [], 0
        for n, last in seqs:
            up = torch.randint(0, 1 << 30, (n,), generator=cpu).tolist()
            depth = []
            for i in range(n):
                parent = i - 1 - up[i] % 4
                depth.append(1 if parent < 0 else depth[parent] + 1)
                if parent >= 0:
                    bits[t + i] = bits[t + parent]
                bits[t + i, i] = 1
            pos += [last + x for x in depth]
            t += n
        word = (bits.view(T, words, 32) << torch.arange(32)).sum(-1)
        s["tree_mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32).cuda()
        s["tree_base"] = torch.tensor([last + 1 for _, last in seqs], dtype=torch.int64).cuda()
        pos = torch.tensor(pos, dtype=torch.int64)
    else:
        pos = torch.cat([torch.arange(last - n + 1, last + 1, dtype=torch.int64) for n, last in seqs])
    s["pos"] = pos.cuda()
    k = case["k"]
    if k:  # each token's chunks: one of each of k strata of the pool, the tail empty where the history has fewer
        rows = (case["rows"] + PAGE - 1) // PAGE * PAGE
        s["cell_pool"] = new(rows // PAGE, PAGE, WIDTH)
        edge = torch.arange(k + 1, device="cuda") * rows // k
        u = torch.rand((T, k), generator=g, device="cuda")
        cells = edge[:-1] + (u * (edge[1:] - edge[:-1])).long().clamp(max=rows // k - 1)
        some = torch.arange(k, device="cuda")[None, :] < (s["pos"] // RATIO)[:, None]
        s["cells"] = torch.where(some, cells, -1).to(torch.int32)
    else:
        s["cell_pool"], s["cells"] = None, None
    return s


def _norm_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H, K, d = case["T"], case["H"], case["K"], case["d"]
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    pages = (T + PAGE - 1) // PAGE + 1
    cells = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T].to(torch.int32)
    fused = 2 * new(T, (H + K) * d)  # the projections' output: a token's query heads, then its key heads
    return dict(q=fused[:, :H * d].view(T, H, d), k=fused[:, H * d:].view(T, K, d), q_gain=1 + 0.1 * new(d),
                k_gain=1 + 0.1 * new(d), pos=case["pos"] - T + 1 + torch.arange(T, device="cuda"),
                k_cell=cells, k_pool=new(pages, PAGE, K * d))


def prepare(case, seed):
    if case["op"] == "qk":
        s = _norm_inputs(case, seed)
        s["q_out"] = torch.empty((case["T"], case["H"], case["d"]), dtype=torch.bfloat16, device="cuda")
    else:
        s = _attention_inputs(case, seed)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    s["case"] = case
    return s


# ------------------------------------------------------------------------------------------------ plain form


def _frequencies(dim):
    """YaRN's NTK-by-parts rotary frequencies, in 64 bits."""
    i = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    theta = ROPE["rope_base"] ** (-2 * i / dim)
    turns = ROPE["rope_orig_len"] * theta / (2 * math.pi)
    keep = ((turns - ROPE["rope_beta_slow"]) / (ROPE["rope_beta_fast"] - ROPE["rope_beta_slow"])).clamp(0, 1)
    return theta * (keep + (1 - keep) / ROPE["rope_factor"])


def _norm_rope(x, gain, angle, rope):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    flat, turned = y[..., :y.shape[-1] - rope], y[..., y.shape[-1] - rope:]
    a, b = turned[..., 0::2], turned[..., 1::2]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([flat, turned], -1).to(torch.bfloat16)


def _norm_plain(s):
    rope = s["case"]["rope"]
    angle = s["pos"].double()[:, None] * _frequencies(rope)[None, :]
    s["q_out"].copy_(_norm_rope(s["q"], s["q_gain"], angle, rope))
    rows = s["k_pool"].view(-1, s["k_pool"].shape[-1])
    rows[s["k_cell"].long()] = _norm_rope(s["k"], s["k_gain"], angle, rope).flatten(1)
    return {"q": s["q_out"], "pool": s["k_pool"]}


def _tokens_seen(s):
    """Slots [T, n] of the cache that each token may see, and which of them it does see."""
    case, pos = s["case"], s["pos"][:, None]
    end = pos if case["op"] == "attn" else s["tree_base"][s["seq"].long()][:, None] - 1
    low = (pos - case["window"] + 1).clamp(min=0)
    window = low + torch.arange(min(case["window"], case["pos"] + 1), device="cuda")
    first = torch.arange(case["first"], device="cuda").expand(pos.shape[0], -1)
    slots, seen = [first, window], [(first < low) & (first <= end), window <= end]
    if case["op"] == "tree":
        bit = torch.arange(32, device="cuda")
        seen.append(((s["tree_mask"].long()[:, :, None] >> bit) & 1).flatten(1).bool())
        slots.append(end + 1 + torch.arange(seen[-1].shape[1], device="cuda"))
    return torch.cat(slots, 1), torch.cat(seen, 1)


def _attention_plain(s):
    slots, seen = _tokens_seen(s)
    width = s["page_table"].shape[1]
    page = s["page_table"][s["seq"].long()].gather(1, (slots // PAGE).clamp(max=width - 1)).long()
    seen = seen & (slots // PAGE < width) & (page >= 0)
    rows = torch.where(seen, page * PAGE + slots % PAGE, 0)
    keys = s["kv_pool"].view(-1, WIDTH)[rows].float()
    if s["cells"] is not None:
        keys = torch.cat([s["cell_pool"].view(-1, WIDTH)[s["cells"].long().clamp(min=0)].float(), keys], 1)
        seen = torch.cat([s["cells"] >= 0, seen], 1)
    score = torch.matmul(s["q"].float(), keys.transpose(1, 2)) * WIDTH ** -0.5
    score = score.masked_fill(~seen[:, None, :], -math.inf)
    top = score.max(-1, keepdim=True).values.clamp(min=-1e30)
    weight = (score - top).exp()
    total = weight.sum(-1, keepdim=True)
    below = total if s["sink_logit"] is None else total + (s["sink_logit"].float()[None, :, None] - top).exp()
    out = torch.matmul(weight, keys) / below.clamp(min=1e-38)
    return {"out": out.to(torch.bfloat16), "lse": (top + total.log())[..., 0]}


def run(s):
    case = s["case"]
    if not own:
        return _norm_plain(s) if case["op"] == "qk" else _attention_plain(s)
    import sparse_attention_kv_c4_gb300 as fm
    if case["op"] == "qk":
        fm.fm_qk_norm_rope(s["pos"], q=s["q"], q_gain=s["q_gain"], q_out=s["q_out"], k=s["k"], k_gain=s["k_gain"],
                           k_pool=s["k_pool"], k_cell=s["k_cell"], rope_dim=case["rope"], eps=EPS, **ROPE)
        return {"q": s["q_out"], "pool": s["k_pool"]}
    if "workspace" not in s:  # a user's program keeps it
        size = fm.fm_csa_attn_workspace(s["q"].shape[0], case["H"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    args = dict(seq=s["seq"], window=case["window"], n_sink=case["first"], cell_pool=s["cell_pool"], cells=s["cells"],
                sink_logit=s["sink_logit"], lse_out=s["lse"], workspace=s["workspace"])
    if case["op"] == "tree":
        fm.fm_csa_attn_tree(s["q"], s["kv_pool"], s["page_table"], s["pos"], s["out"], tree_mask=s["tree_mask"],
                            tree_base=s["tree_base"], **args)
    else:
        fm.fm_csa_attn(s["q"], s["kv_pool"], s["page_table"], s["pos"], s["out"], **args)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------ work, exact values


def work(case):
    if case["op"] == "qk":
        T, n = case["T"], case["T"] * (case["H"] + case["K"]) * case["d"]
        return {"bytes": 4 * n + 4 * case["d"] + 12 * T, "flops": 6 * n}
    T = keys = cells = tokens = 0
    for n, last in _sequences(case):
        T += n
        for p in ([last + 1] * n if case["op"] == "tree" else range(last - n + 1, last + 1)):
            window = min(case["window"], p + 1)
            seen = window + min(case["first"], p + 1 - window)
            chosen = min(case["k"], p // RATIO)
            keys += seen + chosen
            cells += chosen
        tokens += min(last + 1, case["window"] + n + case["first"])
    distinct = min(cells, case["rows"]) + tokens
    return {"bytes": 2 * WIDTH * (2 * T * case["H"] + distinct) + 4 * T * case["H"] + 4 * cells,
            "flops": 4 * WIDTH * case["H"] * keys}


def _exact_rows(x, gain, pos, rope):
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    start = x.shape[-1] - rope
    pair = torch.view_as_complex(y[..., start:].unflatten(-1, (rope // 2, 2)).contiguous())
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * _exact_frequencies(rope))
    y[..., start:] = torch.view_as_real(pair * turn[:, None, :]).flatten(-2)
    return y


def _exact_frequencies(dim):
    values = []
    for i in range(dim // 2):
        theta = ROPE["rope_base"] ** (-2.0 * i / dim)
        ramp = (ROPE["rope_orig_len"] * theta / (2 * math.pi) - ROPE["rope_beta_slow"]) / (ROPE["rope_beta_fast"] - ROPE["rope_beta_slow"])
        ramp = min(1.0, max(0.0, ramp))
        values.append((1 - ramp) * theta / ROPE["rope_factor"] + ramp * theta)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def exact(case, seed):
    if case["op"] == "qk":
        s = _norm_inputs(case, seed)
        pool = s["k_pool"].double()
        pool.view(-1, pool.shape[-1])[s["k_cell"].long()] = _exact_rows(s["k"], s["k_gain"], s["pos"], case["rope"]).flatten(1)
        return {"q": _exact_rows(s["q"], s["q_gain"], s["pos"], case["rope"]), "pool": pool}
    s = _attention_inputs(case, seed)
    T, H = s["q"].shape[:2]
    out = torch.zeros((T, H, WIDTH), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    table = s["page_table"].cpu().numpy()
    seq, pos = s["seq"].tolist(), s["pos"].tolist()
    base = s["tree_base"].tolist() if case["op"] == "tree" else None
    mask = s["tree_mask"].tolist() if case["op"] == "tree" else None
    pool = s["kv_pool"].view(-1, WIDTH)
    chosen = s["cells"].cpu().numpy() if s["cells"] is not None else None
    for t in range(T):
        p, b = pos[t], seq[t]
        low, end = max(0, p - case["window"] + 1), (p if base is None else base[b] - 1)
        slots = list(range(0, min(case["first"], low, end + 1))) + list(range(low, end + 1))
        if base is not None:
            slots += [base[b] + i for i in range(32 * len(mask[t])) if (mask[t][i // 32] >> (i % 32)) & 1]
        rows = [int(table[b, j // PAGE]) * PAGE + j % PAGE for j in slots if table[b, j // PAGE] >= 0]
        keys = pool[torch.tensor(rows, dtype=torch.int64, device="cuda")].double()
        if chosen is not None:
            c = torch.from_numpy(chosen[t][chosen[t] >= 0]).long().cuda()
            keys = torch.cat([keys, s["cell_pool"].view(-1, WIDTH)[c].double()])
        if not len(keys):
            continue
        x = s["q"][t].double() @ keys.T / math.sqrt(WIDTH)
        lse[t] = torch.logsumexp(x, -1)
        z = lse[t] if s["sink_logit"] is None else torch.logaddexp(lse[t], s["sink_logit"].double())
        out[t] = (x - z[:, None]).exp() @ keys
    return {"out": out, "lse": lse}
