"""The operators of the target's verification pass, measured.

A speculative round ends in the target: the drafted rows' keys and values go
into the target's paged cache (`append`), the rows attend over it (`attend`,
bf16 pages or pages of 4-bit values), and the scores of every row are edited by
penalties, biases and a grammar's mask before they are verified (`rules`).

A case is a dict:
  op        "append" | "attend" | "rules"
  streams   streams of the batch
  rows      rows a stream (ragged: between 1 and this many, one stream with none)
and, for append and attend,
  format    "bf16", or "fp4": 4-bit e2m1 values with one e4m3 scale a group of 16
  q, kv, d  query heads, key/value heads, head dimension
  page      slots a page
  lo, hi    committed slots of the streams, spread over [lo, hi]
  window    0, or how far back a row sees; sinks: first slots that stay visible
  mask      "causal" (a row sees its stream's rows up to itself), "block" (all
            of them), "tree" (its ancestors and itself)
for rules
  vocab     scores a row
  grammar   whether a grammar's bit mask applies; bias: biased tokens a stream
  tree      whether the rows are a draft tree's nodes (else a chain)
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    a = dict(op="append", ragged=False)
    t = dict(op="attend", ragged=False, window=0, sinks=0, mask="causal")
    r = dict(op="rules")
    return [
        # one stream's drafted block goes into the cache: the smallest call of a round
        dict(a, name="append block", format="bf16", streams=1, rows=16, q=32, kv=8, d=128, page=64, lo=4096, hi=4096),
        # a prompt pass of several streams, a chunk each
        dict(a, name="append fill", format="bf16", streams=7, rows=1171, q=32, kv=8, d=128, page=64, lo=0, hi=4001,
             ragged=True),
        # the same into a 4-bit cache, forty query heads
        dict(a, name="append fill fp4", format="fp4", streams=8, rows=1024, q=40, kv=8, d=128, page=32, lo=5, hi=9000),
        # one token of one stream
        dict(t, name="token", format="bf16", streams=1, rows=1, q=32, kv=8, d=128, page=64, lo=4096, hi=4096),
        # serving, a token a stream, sliding layers that keep their first slots
        dict(t, name="tokens window", format="bf16", streams=32, rows=1, q=32, kv=8, d=128, page=64, lo=1024,
             hi=16384, window=2048, sinks=4),
        # eight streams' drafted blocks are verified over long contexts
        dict(t, name="blocks", format="bf16", streams=8, rows=16, q=40, kv=8, d=128, page=64, lo=8192, hi=8192),
        # draft trees scored in one pass
        dict(t, name="trees", format="bf16", streams=6, rows=93, q=32, kv=8, d=128, page=16, lo=1000, hi=16001,
             mask="tree"),
        # a chunk of a long prompt
        dict(t, name="fill", format="bf16", streams=1, rows=4096, q=32, kv=8, d=128, page=64, lo=4096, hi=4096),
        # serving from a 4-bit cache, a token a stream
        dict(t, name="tokens fp4", format="fp4", streams=32, rows=1, q=32, kv=8, d=128, page=64, lo=1024, hi=16384),
        # drafted blocks over a 4-bit cache, one stream with nothing to do
        dict(t, name="blocks fp4", format="fp4", streams=9, rows=16, q=40, kv=8, d=128, page=32, lo=4097, hi=16383,
             ragged=True),
        # one stream's drafted block: penalties and a few biased tokens
        dict(r, name="rules block", streams=1, rows=16, vocab=151936, grammar=False, bias=8, tree=False),
        # many streams' trees under grammars
        dict(r, name="rules trees", streams=32, rows=93, vocab=151936, grammar=True, bias=100, tree=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "attend", "rules"))
    if op == "rules":
        c = dict(op=op, streams=_log_int(rng, 1, 48), rows=_log_int(rng, 1, 93), vocab=8 * _log_int(rng, 512, 18992),
                 grammar=rng.random() < 0.5, bias=rng.choice((0, _log_int(rng, 1, 300))), tree=rng.random() < 0.5)
        while c["streams"] * c["rows"] * c["vocab"] > 32 * 93 * 151936:
            c["streams"] = max(1, c["streams"] // 2)
        return c
    kv = rng.choice((1, 2, 4, 8))
    c = dict(op=op, format=rng.choice(("bf16", "fp4")), streams=_log_int(rng, 1, 32), rows=_log_int(rng, 1, 2048),
             q=kv * rng.randint(1, 8), kv=kv, d=rng.choice((64, 128, 128)), page=rng.choice((16, 32, 64, 128)),
             ragged=rng.random() < 0.5)
    c["hi"] = _log_int(rng, 1, 20000)
    c["lo"] = rng.randint(0, c["hi"])
    if op == "append":
        while c["streams"] * c["rows"] * (c["q"] + 2 * c["kv"]) > 8192 * 56:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    c["mask"] = rng.choice(("causal", "causal", "block", "tree"))
    if c["mask"] == "tree":
        c["rows"] = min(c["rows"], 256)
    c["window"] = rng.choice((0, 0, _log_int(rng, 1, 4096)))
    c["sinks"] = rng.choice((0, rng.randint(1, 130))) if c["window"] else 0
    # no more work than the largest listed cases: bytes of the cache, pairs of a row and a slot
    while c["streams"] * c["hi"] * c["kv"] * c["d"] > 8 * 32 * 8192 * 128:
        c["streams"] = max(1, c["streams"] // 2)
    while c["streams"] * c["rows"] * c["q"] * (c["hi"] + c["rows"]) > 4096 * 6144 * 32:
        c["rows"] = max(1, c["rows"] // 2)
    return c


# ---------------------------------------------------------------- shapes: of the case alone


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], uneven, the ends among them."""
    if n == 1:
        return [hi]
    got = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    got[-1] = hi
    return got


def _shape(case):
    """Rows and committed slots of every stream."""
    n, S = case["rows"], case["streams"]
    rows = _spread(S, max(1, n // 2), n) if case.get("ragged") else [n] * S
    if case.get("ragged") and S >= 4:
        rows[1] = 0
    return rows, _spread(S, case["lo"], case["hi"])


def _tree(n):
    """Parents of n nodes, breadth first: four branches, two each below, then chains."""
    parent, level, widths = [-1], [0], [4, 2, 2]
    depth = 0
    while len(parent) < n:
        width = widths[depth] if depth < len(widths) else 1
        depth += 1
        level_next = []
        for p in level:
            for _ in range(width):
                if len(parent) < n:
                    level_next.append(len(parent))
                    parent.append(p)
        level = level_next
    return parent


def _ancestors(parent):
    """bool [n, n]: whether node m is on the path from the root to node r; and the nodes' depths."""
    n = len(parent)
    see = torch.zeros(n, n, dtype=torch.bool)
    depth = torch.zeros(n, dtype=torch.int32)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] = see[p]
            depth[i] = depth[p] + 1
        see[i, i] = True
    return see, depth


def _words(see):
    """Rows of bits as rows of int32 words, bit m of a row in word m / 32."""
    n, m = see.shape
    pad = torch.zeros(n, (m + 31) // 32 * 32, dtype=torch.int64)
    pad[:, :m] = see
    w = (pad.view(n, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def _row_bytes(case):
    return 2 * case["d"] if case["format"] == "bf16" else case["d"] // 2 + case["d"] // 16


def _visible(case):
    """Pairs of a row and a slot that it sees, and slots that some row of their stream sees."""
    rows, lens = _shape(case)
    W, K = case["window"], case["sinks"]
    if case["mask"] == "tree":
        parent = _tree(case["rows"])
        _, depth = _ancestors(parent)
        depth = depth.tolist()
    pairs = slots = 0
    for n, C in zip(rows, lens):
        if n == 0:
            continue
        pos = [C + (depth[j] if case["mask"] == "tree" else j) for j in range(n)]
        first = [max(0, p - W + 1) if W else 0 for p in pos]
        for j in range(n):
            back = first[j]
            ctx = max(0, C - back) + min(K, back, C)
            block = n if case["mask"] == "block" else (depth[j] + 1 if case["mask"] == "tree" else j + 1)
            pairs += ctx + (min(block, W) if W and case["mask"] != "block" else block)
        back = min(first)
        slots += max(0, C - back) + min(K, back, C) + n
    return pairs, slots


def work(case):
    if case["op"] == "rules":
        n = case["streams"] * case["rows"] * case["vocab"]
        return {"bytes": 4.0 * n + 2.0 * case["streams"] * case["vocab"]
                + (n / 8 if case["grammar"] else 0) + 8.0 * case["streams"] * case["bias"], "flops": 5.0 * n}
    rows, lens = _shape(case)
    T, q, kv, d = sum(rows), case["q"], case["kv"], case["d"]
    if case["op"] == "append":
        # the new rows are read and written once, rotated queries too; the angles once a row
        cache = 2 * kv * _row_bytes(case)
        back = 2 * kv * (_row_bytes(case) + 2 * d) if case["format"] == "fp4" else 0  # read back as values
        return {"bytes": float(T * (2 * (q + 2 * kv) * d + 2 * q * d + cache + back + 4 * d)),
                "flops": float(T * 3 * (q + kv) * d)}
    pairs, slots = _visible(case)
    return {"bytes": float(slots * kv * 2 * _row_bytes(case) + 4 * T * q * d), "flops": 4.0 * d * q * pairs}


# ---------------------------------------------------------------- inputs


def _fp4_values():
    v = torch.tensor(E2M1)
    return torch.cat([v, -v])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    s = dict(case=case)
    if case["op"] == "rules":
        S, N, V = case["streams"], case["rows"], case["vocab"]
        s["logits"] = normal(S, N, V, std=4.0)
        # a history of some hundred tokens a stream: part of it prompt (the sign bit), part output (a count)
        s["counts"] = torch.zeros(S, V, dtype=torch.int16, device="cuda")
        seen = torch.randint(0, V, (S, 400), generator=g, device="cuda")
        s["counts"].scatter_(1, seen, torch.randint(1, 6, (S, 400), generator=g, device="cuda").to(torch.int16))
        prompt = torch.randint(0, V, (S, 600), generator=g, device="cuda")
        flag = torch.tensor(-32768, dtype=torch.int16, device="cuda")
        s["counts"].scatter_(1, prompt, s["counts"].gather(1, prompt) | flag)
        # drafted tokens: some of them in the history
        fresh = torch.randint(0, V, (S, N), generator=g, device="cuda")
        old = seen.gather(1, torch.randint(0, 400, (S, N), generator=g, device="cuda"))
        s["tokens"] = torch.where(torch.rand(S, N, generator=g, device="cuda") < 0.5, fresh, old).to(torch.int32)
        parent = _tree(N) if case["tree"] else [i - 1 for i in range(N)]
        see, _ = _ancestors(parent)
        s["path"] = see.to("cuda")
        s["node_mask"] = _words(see).to("cuda").expand(S, N, -1).contiguous() if case["tree"] else None
        s["repetition"] = 1.0 + torch.rand(S, generator=g, device="cuda")
        s["frequency"] = torch.rand(S, generator=g, device="cuda")
        s["presence"] = torch.rand(S, generator=g, device="cuda") - 0.3
        s["bias"] = None
        if case["bias"]:
            b = case["bias"]
            s["bias"] = (torch.arange(S + 1, device="cuda", dtype=torch.int32) * b,
                         torch.randint(0, V, (S * b,), generator=g, device="cuda", dtype=torch.int32),
                         torch.randn(S * b, generator=g, device="cuda") * 5.0)
        s["grammar"] = None
        if case["grammar"]:
            words = (V + 31) // 32
            a, b = (torch.randint(-(2**31), 2**31, (S, N, words), generator=g, device="cuda") for _ in range(2))
            s["grammar"] = (a & b).to(torch.int32)
        return s

    rows, lens = _shape(case)
    S, T, page, kv, d = case["streams"], sum(rows), case["page"], case["kv"], case["d"]
    need = [(C + n + page - 1) // page for C, n in zip(lens, rows)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    # streams' pages lie anywhere in the pool; what a table holds behind a stream's last page is not a page
    at, cols = 0, max(1, max(need))
    s["table"] = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
    for i, n in enumerate(need):
        s["table"][i, :n] = order[at : at + n]
        at += n
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    s["row_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max_rows"] = max(rows)
    s["stream"] = torch.repeat_interleave(torch.arange(S), torch.tensor(rows)).to("cuda")
    s["index"] = torch.cat([torch.arange(n) for n in rows]).to("cuda")
    s["depth"] = s["mask"] = None
    if case["op"] == "attend" and case["mask"] == "tree":
        see, depth = _ancestors(_tree(case["rows"]))
        s["depth"] = depth.to("cuda")[s["index"]]
        s["see"] = see.to("cuda")
        s["mask"] = _words(see).to("cuda")[s["index"]]
    if case["format"] == "bf16":
        s["k"], s["v"] = normal(n_pages, kv, page, d), normal(n_pages, kv, page, d)
        s["k_scale"] = s["v_scale"] = None
    else:
        s["k"], s["v"] = (torch.randint(0, 256, (n_pages, kv, page, d // 2), generator=g, device="cuda",
                                        dtype=torch.uint8) for _ in range(2))
        s["k_scale"], s["v_scale"] = ((0.2 + 0.3 * torch.rand(n_pages, kv, page, d // 16, generator=g, device="cuda")
                                       ).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    s["q"] = normal(T, case["q"], d)
    if case["op"] == "append":
        s["new_k"], s["new_v"] = normal(T, kv, d), normal(T, kv, d)
        pos = torch.arange(max(C + n for C, n in zip(lens, rows)), dtype=torch.float64, device="cuda")
        angle = pos[:, None] * 1.0e6 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    if own:
        import block_diffusion_speculative_tap_gb300 as D

        s["cache"] = D.PagedCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
        s["batch"] = D.Rows(s["row_start"], s["lens"], T, s["max_rows"], s["depth"])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return _rules(s) if op == "rules" else _append(s) if op == "append" else _attend(s)


def _own(s, op):
    c = s["case"]
    if op == "rules":
        import block_diffusion_speculative_tap_gb300 as D

        return D.logit_rules(s["logits"], s["counts"], tokens=s["tokens"], node_mask=s["node_mask"],
                             repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                             bias=s["bias"], grammar=s["grammar"])
    if op == "append":
        q = s["cache"].append(s["batch"], s["new_k"], s["new_v"], s["rope"], q=s["q"])
        if c["format"] == "bf16":
            return q, s["k"], s["v"]
        return (q, *s["cache"].read(s["batch"]))
    return s["cache"].attend(s["batch"], s["q"], window=c["window"], sinks=c["sinks"],
                             mask=s["mask"] if c["mask"] == "tree" else c["mask"])


def _rotate(x, cos, sin):
    """Rotate-half: the pair (i, i + d/2) by the angle of the row's position."""
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)


def _quantise(x):
    """Groups of 16: scale = e4m3(max / 6), values to the nearest e2m1 (ties to the even code)."""
    x = x.float().unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    y = torch.where(s > 0, x / s, torch.zeros_like(x))
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(x)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scale):
    """The values, in 32 bits, that 4-bit codes and their scales stand for."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    v = _fp4_values().to(codes.device)[code].unflatten(-1, (-1, 16))
    return (v * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _append(s):
    c = s["case"]
    pos = (s["lens"][s["stream"]] + s["index"]).long()
    page = s["table"][s["stream"], pos // c["page"]].long()
    slot = pos % c["page"]
    cos, sin = s["rope"][pos][:, None].unbind(-1)
    q, k, v = _rotate(s["q"], cos, sin), _rotate(s["new_k"], cos, sin), s["new_v"]
    if c["format"] == "bf16":
        s["k"][page, :, slot] = k
        s["v"][page, :, slot] = v
        return q, s["k"], s["v"]
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    s["k"][page, :, slot], s["v"][page, :, slot] = kc, vc
    s["k_scale"][page, :, slot], s["v_scale"][page, :, slot] = ks, vs
    return (q, _values(s["k"][page, :, slot], s["k_scale"][page, :, slot]).to(torch.bfloat16),
            _values(s["v"][page, :, slot], s["v_scale"][page, :, slot]).to(torch.bfloat16))


def _see(s, L):
    """bool [S, R, L]: whether row r of a stream sees its slot."""
    c = s["case"]
    R = s["max_rows"]
    C = s["lens"].long()[:, None, None]
    slot = torch.arange(L, device="cuda")[None, None]
    r = torch.arange(R, device="cuda")[None, :, None]
    n = (s["row_start"][1:] - s["row_start"][:-1]).long()[:, None, None]
    m = (slot - C).clamp(0, R - 1)  # a slot's row
    if c["mask"] == "tree":
        depth = _ancestors(_tree(c["rows"]))[1].to("cuda").long()[:R]
        block = s["see"][:R, :R][r, m]
        pos, at = C + depth[r], torch.where(slot < C, slot, C + depth[m])
    else:
        block = (m <= r) if c["mask"] == "causal" else torch.ones_like(m <= r)
        pos, at = C + r, slot
    see = torch.where(slot < C, torch.ones_like(block), block & (slot < C + n)) & (r < n)
    if c["window"]:
        see = see & ((pos - at < c["window"]) | (slot < c["sinks"]))
    return see


def _attend(s):
    c = s["case"]
    S, R, kv, d = c["streams"], s["max_rows"], c["kv"], c["d"]
    pages = s["table"].long().clamp(min=0)
    if c["format"] == "bf16":
        k, v = s["k"][pages].float(), s["v"][pages].float()
    else:
        k, v = _values(s["k"][pages], s["k_scale"][pages]), _values(s["v"][pages], s["v_scale"][pages])
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))  # [S, kv, L, d]
    L = k.shape[2]
    see = _see(s, L)
    used = see.any(1)[:, None, :, None]
    v = torch.where(used, v, torch.zeros_like(v))
    q = torch.zeros(S, R, c["q"], d, device="cuda")
    q[s["stream"], s["index"]] = s["q"].float()
    q = q.unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)  # [S, kv, G, R, d]
    G = q.shape[2]
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (G, R)) * d**-0.5
    see = see[:, None, None]
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))))
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.flatten(2, 3), v).unflatten(2, (G, R)) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[s["stream"], s["index"]].to(torch.bfloat16)


def _rules(s):
    S, N, V = s["logits"].shape
    x = s["logits"].float()
    c = s["counts"].int()
    prompt, count = c < 0, (c & 0x7FFF).float()
    # each row's own path (the root, the last committed token, is in the counts)
    see = s["path"].clone()
    see[:, 0] = False
    row, node = see.nonzero(as_tuple=True)
    extra = torch.zeros(S, N, V, device="cuda")
    b = torch.arange(S, device="cuda")[:, None].expand(S, row.numel())
    extra.index_put_((b, row.expand(S, -1), s["tokens"].long()[:, node]), torch.ones((), device="cuda"), accumulate=True)
    count = extra.add_(count[:, None])
    rep, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    seen = (count > 0) | prompt[:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count - pres * (count > 0).float()
    if s["bias"] is not None:
        start, ids, vals = s["bias"]
        who = torch.repeat_interleave(torch.arange(S, device="cuda"), ids.numel() // S)
        add = torch.zeros(S, V, device="cuda", dtype=torch.float64)
        add.index_put_((who, ids.long()), vals.double(), accumulate=True)
        x = x + add.float()[:, None]
    if s["grammar"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        may = ((s["grammar"][..., None] >> bit) & 1).flatten(2)[..., :V].bool()
        x = torch.where(may, x, torch.full((), -math.inf, device="cuda"))
    return x.to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rules":
        return _exact_rules(s)
    rows, lens = _shape(case)
    start = s["row_start"].tolist()
    page, d, kv = case["page"], case["d"], case["kv"]

    def slots(i, n):
        p = torch.arange(n, device="cuda")
        return s["table"][i, p // page].long(), p % page

    if case["op"] == "append":
        angle = 1.0e6 ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)

        def turned(x, pos):
            a = torch.view_as_complex(torch.stack([x[..., : d // 2].double(), x[..., d // 2 :].double()], -1))
            t = pos.double()[:, None, None] * angle
            a = a * torch.complex(torch.cos(t).float().double(), torch.sin(t).float().double())
            return torch.cat([a.real, a.imag], -1)

        q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        k = torch.empty(s["new_k"].shape, dtype=torch.float64, device="cuda")
        for i, (n, C) in enumerate(zip(rows, lens)):
            at = slice(start[i], start[i] + n)
            pos = torch.arange(C, C + n, device="cuda")
            q[at], k[at] = turned(s["q"][at], pos), turned(s["new_k"][at], pos)
        if case["format"] == "fp4":
            return [q, _nearest_fp4(k), _nearest_fp4(s["new_v"].double())]
        pool_k, pool_v = s["k"].double(), s["v"].double()
        for i, (n, C) in enumerate(zip(rows, lens)):
            pages, at = slots(i, C + n)
            pool_k[pages[C:], :, at[C:]] = k[start[i] : start[i] + n]
            pool_v[pages[C:], :, at[C:]] = s["new_v"][start[i] : start[i] + n].double()
        return [q, pool_k, pool_v]

    pairs, _ = _visible(case)
    if pairs * case["q"] * d > 3.5e11:  # 64-bit products are slow here
        return None

    def values(x, scale, i, n):
        pages, at = slots(i, n)
        if scale is None:
            return x[pages, :, at].double()
        c = x[pages, :, at].long()
        c = torch.stack([c % 16, c // 16], -1).reshape(n, kv, d)
        mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[c % 8] * (1 - 2 * (c // 8))
        return mag * scale[pages, :, at].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (n, C) in enumerate(zip(rows, lens)):
        k, v = values(s["k"], s["k_scale"], i, C + n), values(s["v"], s["v_scale"], i, C + n)
        for j0 in range(0, n, 256):  # a part of the rows at a time
            j = torch.arange(j0, min(n, j0 + 256), device="cuda")
            t = torch.arange(C + n, device="cuda")
            p, at = C + j, t
            see = t[None] <= p[:, None]
            if case["mask"] == "block":
                see = torch.ones_like(see)
            if case["mask"] == "tree":
                parent = _tree(case["rows"])
                anc, depth = _ancestors(parent)
                see = torch.cat([torch.ones(len(j), C, dtype=torch.bool), anc[j.cpu(), :n]], 1).cuda()
                p, at = C + depth[j.cpu()].cuda(), torch.cat([t[:C], C + depth[:n].cuda()])
            if case["window"]:
                see &= (at[None] > p[:, None] - case["window"]) | (t[None] < case["sinks"])
            qi = s["q"][start[i] + j0 : start[i] + j0 + len(j)].double().view(len(j), kv, -1, d)
            x = torch.einsum("rhgd,thd->hgrt", qi, k) / math.sqrt(d)
            w = torch.softmax(x.masked_fill(~see, -math.inf), -1)
            out[start[i] + j0 : start[i] + j0 + len(j)] = torch.einsum("hgrt,thd->rhgd", w, v).reshape(len(j), -1, d)
    return out


def _nearest_fp4(k):
    """The 4-bit values of what a bf16 cache would hold, by the nearest of the sixteen."""
    k = k.to(torch.bfloat16).double()
    g = k.reshape(*k.shape[:-1], -1, 16)
    top = g.abs().amax(-1) / 6
    e4m3 = torch.arange(127, dtype=torch.uint8, device=k.device).view(torch.float8_e4m3fn).double()
    i = torch.searchsorted(e4m3, top.clamp(max=448.0)).clamp(1, 126)
    lo, hi = e4m3[i - 1], e4m3[i]
    up = (top - lo > hi - top) | ((top - lo == hi - top) & (i % 2 == 0))
    scale = torch.where(up, hi, lo)[..., None]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=k.device)
    x = torch.where(scale > 0, g.abs() / scale, torch.zeros_like(g)).clamp(max=6.0)
    j = torch.searchsorted(grid, x).clamp(1, 7)
    a, b = grid[j - 1], grid[j]
    up = (x - a > b - x) | ((x - a == b - x) & (j % 2 == 0))
    return (torch.where(up, b, a) * scale * torch.sign(g)).reshape(k.shape)


def _exact_rules(s):
    S, N, V = s["logits"].shape
    if S * N * V > 2**29:  # twenty seconds' worth
        return None
    out = s["logits"].double()
    see, tokens = s["path"].cpu(), s["tokens"].long()
    for i in range(S):
        c = s["counts"][i].long() & 0xFFFF
        for n in range(N):
            path = [m for m in range(1, N) if see[n, m]]
            count = (c % 32768) + torch.bincount(tokens[i][path], minlength=V)
            x = out[i, n]
            again = (count > 0) | (c >= 32768)
            r = s["repetition"][i].double()
            x = torch.where(again, torch.where(x > 0, x / r, x * r), x)
            x = x - s["frequency"][i].double() * count - s["presence"][i].double() * (count > 0)
            if s["bias"] is not None:
                b = slice(int(s["bias"][0][i]), int(s["bias"][0][i + 1]))
                x = x.index_add(0, s["bias"][1][b].long(), s["bias"][2][b].double())
            if s["grammar"] is not None:
                ids = torch.arange(V, device="cuda")
                x = torch.where((s["grammar"][i, n].long()[ids // 32] >> (ids % 32)) & 1 == 1, x, -math.inf)
            out[i, n] = x
    return out
