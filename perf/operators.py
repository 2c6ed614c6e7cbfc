"""The operators around attention, as workloads: what a pass reads, computes and returns.

Five operators: queries and keys normalised per head and rotated by position (`norm`), the gradient
of that (`grad`), the same pass writing keys and values into a paged cache (`write`), the bookkeeping
of that cache (`pages`), and decode for sequences that share a long prefix (`decode`).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, through the library's entry point.  ``exact`` computes it from its definition in 64
bits.  A case is a dict of plain values; lengths of a ragged batch follow from the case alone, so
that ``work`` can count them, and everything else is drawn from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------
def listed():
    return [
        # a training batch between the fused projection and the causal attention over 8192 tokens
        {"name": "norm_train_2x8192", "op": "norm", "dtype": "bf16", "B": 2, "N": 8192, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "axes": 1, "interleaved": False},
        # an image encoder's tokens: one odd-sized grid, three position axes, 32-bit heads of 64
        {"name": "norm_image_f32_1025", "op": "norm", "dtype": "f32", "B": 1, "N": 1025, "Hq": 16, "Hkv": 16,
         "d": 64, "rot": 64, "axes": 3, "interleaved": False},
        # the backward pass of a training batch of the causal n = 2048 size
        {"name": "grad_train_4x2048", "op": "grad", "dtype": "bf16", "B": 4, "N": 2048, "Hq": 16, "Hkv": 16,
         "d": 128, "rot": 128, "axes": 1, "interleaved": False},
        # the backward pass over video tokens: grouped heads, three axes, pairs side by side, half of
        # each head rotated, an odd count of tokens
        {"name": "grad_video_grouped_5003", "op": "grad", "dtype": "bf16", "B": 1, "N": 5003, "Hq": 32, "Hkv": 4,
         "d": 128, "rot": 64, "axes": 3, "interleaved": True},
        # one decode step of 64 sequences: a token each into the cache
        {"name": "write_step_64", "op": "write", "T": 64, "pad": 0, "Hq": 32, "Hkv": 8, "page": 16, "rot": 128, "axes": 1},
        # a prompt chunk of several requests, padded to a fixed token count
        {"name": "write_prompt_16384", "op": "write", "T": 16384, "pad": 301, "Hq": 32, "Hkv": 8, "page": 64, "rot": 128,
         "axes": 1},
        # the pages of one decode step of 64 sequences
        {"name": "pages_step_64", "op": "pages", "B": 64, "page": 16, "longest": 32768, "prompt": 0, "ended": 2},
        # many requests at once: decode steps, fresh prompts and ended requests mixed
        {"name": "pages_mixed_2000", "op": "pages", "B": 2000, "page": 16, "longest": 4096, "prompt": 500, "ended": 61},
        # few users behind one short system prompt, where latency counts
        {"name": "decode_few_b4_p700", "op": "decode", "B": 4, "Hq": 32, "Hkv": 8, "groups": 1, "prefix": 700,
         "own": 90, "page": 16},
        # a serving batch behind one document of 32768 tokens
        {"name": "decode_doc_b64_p32768", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "groups": 1, "prefix": 32768,
         "own": 400, "page": 16},
        # several prompts of different lengths, some sequences with none, some with nothing of their own
        {"name": "decode_groups_b97_p6001", "op": "decode", "B": 97, "Hq": 32, "Hkv": 4, "groups": 5, "prefix": 6001,
         "own": 1000, "page": 64},
        # the largest: a sampling batch of 256 answers to one long prompt, well into their answers
        {"name": "decode_sampling_b256_p16384", "op": "decode", "B": 256, "Hq": 32, "Hkv": 8, "groups": 1,
         "prefix": 16384, "own": 1500, "page": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "grad", "write", "pages", "decode", "decode"])
    if op in ("norm", "grad"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "B": rng.randint(1, 3),
                "N": _log(rng, 1, 3000), "Hq": hkv * rng.choice([1, 2, 3, 4]), "Hkv": hkv, "d": d,
                "rot": rng.choice([0, 32, d // 2, d, d]), "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.random() < 0.4}
    if op == "write":
        t = _log(rng, 1, 12000)
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "T": t, "pad": rng.randint(0, min(t - 1, 200)), "Hq": hkv * rng.choice([1, 2, 4, 8]),
                "Hkv": hkv, "page": rng.choice([8, 16, 32, 64, 128]), "rot": rng.choice([64, 96, 128, 128]),
                "axes": rng.choice([1, 1, 3])}
    if op == "pages":
        b = _log(rng, 1, 1900)
        p = rng.randint(0, b // 3)
        return {"op": op, "B": b, "page": rng.choice([8, 16, 32, 64, 128]), "longest": _log(rng, 64, 4000), "prompt": p,
                "ended": rng.randint(0, b // 4)}
    hkv = rng.choice([1, 2, 4, 8])
    b = _log(rng, 1, 200)
    return {"op": op, "B": b, "Hq": hkv * rng.choice([1, 2, 4, 8]), "Hkv": hkv, "groups": rng.randint(1, min(b, 6)),
            "prefix": _log(rng, 20, 12000), "own": _log(rng, 4, 1200), "page": rng.choice([8, 16, 32, 64, 128, 256])}


# what follows from a case alone -----------------------------------------------------------------
def _sections(rot, axes):
    """Rotated pairs of each axis: uneven, as models split them."""
    if axes == 1:
        return None
    pairs = rot // 2
    first = pairs // 4
    if axes == 2:
        return [first, pairs - first]
    second = (pairs - first) // 2
    return [first, second, pairs - first - second]


def _groups(case):
    """(first sequence of each group and the end of the last, prefix length of each group)."""
    rng = random.Random("groups %(B)d %(groups)d %(prefix)d" % case)
    B, n = case["B"], case["groups"]
    if n == 1:
        return [0, B], [case["prefix"]]
    cuts = sorted(rng.sample(range(1, B), n - 1)) if B > n else list(range(1, n))
    starts = [0] + cuts + [max(B - 1, cuts[-1])]  # the last sequence is in no group where there is room
    lens = [rng.randint(1, case["prefix"]) for _ in range(n)]
    lens[rng.randrange(n)] = case["prefix"]
    return starts, lens


def _own_lens(case):
    rng = random.Random("own %(B)d %(own)d" % case)
    lens = [rng.randint(1, case["own"]) for _ in range(case["B"])]
    if case["B"] > 8:
        lens[3], lens[5] = 0, case["own"]
    return lens


def _requests(case):
    """Lengths before and after the step."""
    rng = random.Random("requests %(B)d %(longest)d %(prompt)d" % case)
    old, new = [], []
    for b in range(case["B"]):
        if b < case["prompt"]:
            old.append(0)
            new.append(rng.randint(1, max(1, case["longest"] // 8)))
        elif b < case["prompt"] + case["ended"]:
            old.append(rng.randint(1, case["longest"]))
            new.append(0)
        else:
            n = rng.randint(1, case["longest"] - 1)
            old.append(n)
            new.append(n + 1)
    order = list(range(case["B"]))
    rng.shuffle(order)
    return [old[i] for i in order], [new[i] for i in order]


def _ceil(a, b):
    return -(-a // b)


def _max_pos(case):
    if case["op"] == "write":
        return 32768
    return case["N"] if case["axes"] == 1 else 128


def work(case):
    op = case["op"]
    if op in ("norm", "grad"):
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hkv"])
        size = 2 if case["dtype"] == "bf16" else 4
        tokens = case["B"] * case["N"] if case["axes"] > 1 else case["N"]
        table = min(tokens, _max_pos(case)) * case["rot"] * 4
        n = rows * case["d"]
        return {"bytes": n * size * (2 if op == "norm" else 3) + table + tokens * 4 * case["axes"],
                "flops": n * (7 if op == "norm" else 16)}
    if op == "write":
        live = case["T"] - case["pad"]
        return {"bytes": live * 2 * 128 * 2 * (case["Hq"] + 2 * case["Hkv"]) + live * 4 * (1 + case["axes"])
                + min(live, 32768) * case["rot"] * 4, "flops": live * 7 * 128 * (case["Hq"] + case["Hkv"])}
    if op == "pages":
        old, new = _requests(case)
        tokens = sum(max(n - o, 0) for o, n in zip(old, new))
        moved = sum(abs(_ceil(n, case["page"]) - _ceil(o, case["page"])) for o, n in zip(old, new))
        return {"bytes": 12 * case["B"] + 8 * tokens + 8 * moved, "flops": 0}
    starts, plens = _groups(case)
    own_lens = _own_lens(case)
    keys = sum(plens) + sum(own_lens)
    pairs = sum((b - a) * n for a, b, n in zip(starts, starts[1:], plens)) + sum(own_lens)
    return {"bytes": keys * case["Hkv"] * 512 + case["B"] * case["Hq"] * (512 + 4) + 4 * _ceil(keys, case["page"]),
            "flops": pairs * case["Hq"] * 512}


# ----------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------
def _rope_table(max_pos, rot):
    pairs = max(rot // 2, 1)
    freq = 1e6 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * freq[None, : rot // 2]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _weight(g, d, dtype):
    return (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype)


def _positions(case, g, tokens):
    """Positions of a run of tokens: counted up, or frame, row and column of a grid."""
    if case["axes"] == 1:
        return torch.arange(tokens, device=DEV, dtype=torch.int32)
    t = torch.arange(tokens, device=DEV, dtype=torch.int32)
    width = max(1, min(32, int(math.isqrt(tokens))))
    at = int(torch.randint(0, 32, (1,), generator=g, device=DEV))
    grid = [at + (t // (width * width)) % 64, at + (t // width) % width, at + t % width]
    return torch.stack(grid[: case["axes"]]).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"norm": _prepare_norm, "grad": _prepare_norm, "write": _prepare_write, "pages": _prepare_pages,
            "decode": _prepare_decode}[case["op"]](case, g)


def _prepare_norm(case, g):
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, N, Hq, Hkv, d = (case[n] for n in ("B", "N", "Hq", "Hkv", "d"))
    # the projection's output: queries, keys and values of a token side by side
    qkv = _normal(g, B, N, Hq + 2 * Hkv, d, dtype=dt, scale=1.7)
    s = dict(case)
    s["q"] = qkv[:, :, :Hq].transpose(1, 2)
    s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    s["wq"], s["wk"] = _weight(g, d, dt), _weight(g, d, dt)
    s["rope"] = _rope_table(_max_pos(case), case["rot"])
    s["positions"] = _positions(case, g, N)
    s["sections"] = _sections(case["rot"], case["axes"])
    if case["op"] == "grad":
        s["dq_out"] = _normal(g, B, Hq, N, d, dtype=dt)
        s["dk_out"] = _normal(g, B, Hkv, N, d, dtype=dt)
    return s


def _prepare_write(case, g):
    T, Hq, Hkv, page, live = case["T"], case["Hq"], case["Hkv"], case["page"], case["T"] - case["pad"]
    qkv = _normal(g, T, Hq + 2 * Hkv, 128, scale=1.7)
    s = dict(case)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["wq"], s["wk"] = _weight(g, 128, torch.bfloat16), _weight(g, 128, torch.bfloat16)
    s["rope"] = _rope_table(32768, case["rot"])
    s["sections"] = _sections(case["rot"], case["axes"])
    pos = torch.randint(0, 32768, (1 if case["axes"] == 1 else case["axes"], T), generator=g, device=DEV, dtype=torch.int32)
    s["positions"] = pos[0] if case["axes"] == 1 else pos
    pages = _ceil(T, page) + 7
    order = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    slots = order[t // page] * page + t % page
    s["slots"] = torch.where(t < live, slots, torch.full_like(slots, -1)).int()
    s["k_cache"] = torch.zeros(pages, page, Hkv, 128, device=DEV, dtype=torch.bfloat16)
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    s["q_out"] = torch.zeros(T, Hq, 128, device=DEV, dtype=torch.bfloat16)
    return s


def _prepare_pages(case, g):
    old, new = _requests(case)
    ps = case["page"]
    had, need = [_ceil(n, ps) for n in old], [_ceil(n, ps) for n in new]
    spare = sum(max(n - h, 0) for h, n in zip(had, need)) + 100
    total = sum(had) + spare
    max_pages = _ceil(case["longest"], ps)
    order = torch.randperm(total, generator=g, device=DEV).int()
    s = dict(case)
    table = torch.full((case["B"], max_pages), -1, device=DEV, dtype=torch.int32)
    i = torch.arange(max_pages, device=DEV)[None]
    h = torch.tensor(had, device=DEV)[:, None]
    at = (h.cumsum(0) - h) + i
    s["block_table"] = torch.where(i < h, order[at.clamp(max=total - 1)], table).contiguous()
    head = int(torch.randint(0, 1 << 40, (1,), generator=g, device=DEV))
    ring = torch.full((total,), -1, device=DEV, dtype=torch.int32)
    ring[(head + torch.arange(spare, device=DEV)) % total] = order[sum(had):]
    s["free_pages"] = ring
    s["ring"] = torch.tensor([head, head + spare, 0], device=DEV, dtype=torch.int64)
    s["old_lens"] = torch.tensor(old, device=DEV, dtype=torch.int32)
    s["new_lens"] = torch.tensor(new, device=DEV, dtype=torch.int32)
    s["offset"] = torch.randint(0, 5000, (case["B"],), generator=g, device=DEV, dtype=torch.int32)
    tokens = sum(max(n - o, 0) for o, n in zip(old, new))
    s["max_tokens"] = _ceil(tokens + 1, 64) * 64
    return s


def _prepare_decode(case, g):
    B, Hq, Hkv, ps = case["B"], case["Hq"], case["Hkv"], case["page"]
    starts, plens = _groups(case)
    own_lens = _own_lens(case)
    need = [_ceil(n, ps) for n in plens + own_lens]
    pages = sum(need) + 5
    s = dict(case)
    s["starts"], s["plens"], s["own_lens"] = starts, plens, own_lens
    s["q"] = _normal(g, B, Hq, 1, 128, scale=1.3)
    s["k_cache"] = _normal(g, pages, ps, Hkv, 128)
    s["v_cache"] = _normal(g, pages, ps, Hkv, 128)
    order = torch.randperm(pages, generator=g, device=DEV).int()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n])
        at += n

    def table(part):
        width = max(1, max(len(r) for r in part))
        t = torch.full((len(part), width), -1, device=DEV, dtype=torch.int32)
        for i, r in enumerate(part):
            t[i, : len(r)] = r
        return t

    s["prefix_table"], s["block_table"] = table(rows[: len(plens)]), table(rows[len(plens):])
    s["prefix_lens"] = torch.tensor(plens, device=DEV, dtype=torch.int32)
    s["group_starts"] = torch.tensor(starts, device=DEV, dtype=torch.int32)
    s["seq_lens"] = torch.tensor(own_lens, device=DEV, dtype=torch.int32)
    return s


# ----------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# plain forms ----------------------------------------------------------------------------------
def _pair_axis(sections, pairs, device):
    axis = torch.zeros(pairs, dtype=torch.long, device=device)
    for at in list(torch.tensor(sections or [pairs]).cumsum(0).tolist())[:-1]:
        axis += (torch.arange(pairs, device=device) >= at).long()
    return axis


def _angles(s, dtype):
    """cos and sin [tokens, rot / 2] of every rotated pair."""
    pairs = s["rot"] // 2
    col = torch.arange(pairs, device=DEV)
    pos = s["positions"].long()
    rows = pos[:, None].expand(-1, pairs) if pos.dim() == 1 else pos[_pair_axis(s["sections"], pairs, DEV)].t()
    table = s["rope"].to(dtype)
    return table[rows, col], table[rows, col + pairs]


def _rotate(y, cos, sin, rot, interleaved):
    """y [..., tokens, d], cos and sin [tokens, rot / 2]."""
    z = y.clone()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z[..., lo] = y[..., lo] * cos - y[..., hi] * sin
    z[..., hi] = y[..., hi] * cos + y[..., lo] * sin
    return z


EPS = 1e-6


def _norm_rope(x, w, cos, sin, rot, interleaved):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, cos, sin, rot, interleaved).to(x.dtype)


def _plain_norm(s):
    cos, sin = _angles(s, torch.float32)
    return tuple(_norm_rope(s[x], s["w" + x], cos, sin, s["rot"], s["interleaved"]).contiguous() for x in "qk")


def _plain_grad(s):
    cos, sin = _angles(s, torch.float32)
    dx, dw = [], []
    for n in "qk":
        x, w = s[n].float(), s["w" + n].float()
        dy = _rotate(s["d%s_out" % n].float(), cos, -sin, s["rot"], s["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dw.append((dy * xh).sum((0, 1, 2)))
        gw = dy * w
        dx.append((r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(s[n].dtype))
    return dx[0], dx[1], dw[0], dw[1]


def _plain_write(s):
    cos, sin = _angles(s, torch.float32)
    live = s["slots"] >= 0
    q, k = (_norm_rope(s[n].transpose(0, 1), s["w" + n], cos, sin, s["rot"], False).transpose(0, 1) for n in "qk")
    s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
    n = s["T"] - s["pad"]  # the tokens that have a slot come first
    slots = s["slots"][:n].long()
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], s["v"])):
        cache.view(-1, *cache.shape[2:])[slots] = rows[:n]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_pages(s):
    ps, cap, table = s["page"], s["free_pages"].numel(), s["block_table"]
    old, new = s["old_lens"].long(), s["new_lens"].long()
    had, need = (old + ps - 1) // ps, (new + ps - 1) // ps
    grow, shrink, count = (need - had).clamp(min=0), (had - need).clamp(min=0), (new - old).clamp(min=0)
    g0, s0, t1 = grow.cumsum(0) - grow, shrink.cumsum(0) - shrink, count.cumsum(0)
    head, tail = s["ring"][0], s["ring"][1]
    i = torch.arange(table.shape[1], device=DEV)[None]
    h, n = had[:, None], need[:, None]
    taken = s["free_pages"][(head + g0[:, None] + i - h).clamp(min=0) % cap]
    given = (i >= n) & (i < h)
    at = torch.where(given, (tail + s0[:, None] + i - n) % cap, cap)
    ring = torch.cat([s["free_pages"], s["free_pages"][:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:cap]
    s["free_pages"].copy_(ring)
    table.copy_(torch.where((i >= h) & (i < n), taken, table))
    cu = torch.cat([t1.new_zeros(1), t1])
    t = torch.arange(s["max_tokens"], device=DEV)
    live = t < cu[-1]
    b = torch.searchsorted(t1, t, right=True).clamp(max=len(old) - 1)
    p = torch.where(live, old[b] + t - cu[b], 0)
    slots = torch.where(live, table[b, p // ps] * ps + p % ps, -1)
    positions = torch.where(live, p + s["offset"][b], 0)
    ring_out = torch.stack([head + grow.sum(), tail + shrink.sum(), torch.zeros_like(head)])
    return table, s["free_pages"], ring_out, cu.int(), slots.int(), positions.int()


def _partial(q, k, v, hidden):
    """Softmax attention of q [..., rows, d] over k, v [..., keys, d], as (max, sum, weighted values)."""
    x = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(128))
    if hidden is not None:
        x = x.masked_fill(hidden, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = (x - m).exp()
    return m, e.sum(-1, keepdim=True), e @ v


def _plain_decode(s):
    B, Hq, Hkv, ps = s["B"], s["Hq"], s["Hkv"], s["page"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, 128)

    def keys(cache, pages, n):  # [..., pages] -> [..., Hkv, n, d]
        rows = cache[pages.long().clamp(min=0)].flatten(-4, -3)[..., :n, :, :]
        return rows.transpose(-3, -2).float()

    n = max(max(s["own_lens"]), 1)
    hidden = torch.arange(n, device=DEV)[None] >= s["seq_lens"][:, None]
    m, l, o = _partial(q, keys(s["k_cache"], s["block_table"], n), keys(s["v_cache"], s["block_table"], n).masked_fill(
        hidden[:, None, :, None], 0), hidden[:, None, None])
    for i, (a, b, n) in enumerate(zip(s["starts"], s["starts"][1:], s["plens"])):
        if b > a:
            pages = s["prefix_table"][i, : _ceil(n, ps)]
            rows = q[a:b].transpose(0, 1).flatten(1, 2)  # [Hkv, sequences x group, d]
            part = _partial(rows, keys(s["k_cache"], pages, n), keys(s["v_cache"], pages, n), None)
            pm, pl, po = (x.view(Hkv, b - a, -1, x.shape[-1]).transpose(0, 1) for x in part)
            top = torch.maximum(m[a:b], pm)
            f, pf = (m[a:b] - top).exp(), (pm - top).exp()
            m[a:b], l[a:b], o[a:b] = top, l[a:b] * f + pl * pf, o[a:b] * f + po * pf
    out = torch.where(l > 0, o / l, 0).to(s["q"].dtype).view(B, Hq, 1, 128)
    return out, torch.where(l > 0, m + l.log(), -math.inf).view(B, Hq)


_PLAIN = {"norm": _plain_norm, "grad": _plain_grad, "write": _plain_write, "pages": _plain_pages, "decode": _plain_decode}


# the library's entry points ---------------------------------------------------------------------
def _own_norm(s):
    from exact_io_aware_82_b200 import attn_qk_norm_rope

    return attn_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], s["positions"], sections=s["sections"],
                             interleaved=s["interleaved"], eps=EPS)


def _own_grad(s):
    from exact_io_aware_82_b200 import attn_qk_norm_rope_bwd

    return attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["wq"], s["wk"], s["rope"], s["positions"],
                                 sections=s["sections"], interleaved=s["interleaved"], eps=EPS)


def _own_write(s):
    from exact_io_aware_82_b200 import attn_qk_norm_rope_paged

    q = attn_qk_norm_rope_paged(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["rope"], s["positions"], s["slots"],
                                s["k_cache"], s["v_cache"], sections=s["sections"], eps=EPS, q_out=s["q_out"])
    return q, s["k_cache"], s["v_cache"]


def _own_pages(s):
    from exact_io_aware_82_b200 import attn_page_update

    ring, cu, slots, positions = attn_page_update(s["block_table"], s["old_lens"], s["new_lens"], s["free_pages"], s["ring"],
                                                  s["page"], s["max_tokens"], pos_offset=s["offset"])
    return s["block_table"], s["free_pages"], ring, cu, slots, positions


def _own_decode(s):
    from exact_io_aware_82_b200 import attn_decode_shared_prefix

    return attn_decode_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"],
                                     s["group_starts"], s["block_table"], s["seq_lens"], max(s["plens"]),
                                     max(max(s["own_lens"]), 1))


_OWN = {"norm": _own_norm, "grad": _own_grad, "write": _own_write, "pages": _own_pages, "decode": _own_decode}


# ----------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ----------------------------------------------------------------------------------------------
def _exact_matrix(s):
    """For every token the rotation of a whole head as (diagonal, partner, partner's factor): column j of
    the result is diag[j] * y[j] + off[j] * y[partner[j]]."""
    rot, pairs, d = s["rot"], s["rot"] // 2, s.get("d", 128)
    sections = s["sections"] or [pairs]
    pos = s["positions"].reshape(-1, s["positions"].shape[-1]).cpu().tolist()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    j = torch.arange(d, device=DEV)
    if s.get("interleaved"):
        pair, first, partner = j // 2, j % 2 == 0, j ^ 1
    else:
        pair, first = j % max(pairs, 1), j < pairs
        partner = torch.where(first, j + pairs, j - pairs)
    inside = j < rot
    partner = torch.where(inside, partner, j)
    diag = torch.ones(len(pos[0]), d, device=DEV, dtype=torch.float64)
    off = torch.zeros_like(diag)
    rows = torch.tensor(pos, device=DEV)
    for c in range(rot):
        i = int(pair[c])
        at = rows[axis[i]]
        diag[:, c] = s["rope"][at, i].double()
        off[:, c] = s["rope"][at, pairs + i].double() * (-1.0 if bool(first[c]) else 1.0)
    return diag, off, partner


def _exact_rows(x, w, diag, off, partner):
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    return diag * y + off * y[..., partner]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        return None  # whole numbers
    if op == "decode":
        return _exact_decode(s)
    diag, off, partner = _exact_matrix(s)
    if op == "norm":
        return tuple(_exact_rows(s[n], s["w" + n], diag, off, partner) for n in "qk")
    if op == "write":
        out = [s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()]
        live = s["slots"] >= 0
        at = s["slots"][live].long()
        q, k = (_exact_rows(s[n].transpose(0, 1), s["w" + n], diag, off, partner).transpose(0, 1) for n in "qk")
        out[0][live] = q[live]
        out[1].view(-1, s["Hkv"], 128)[at] = k[live]
        out[2].view(-1, s["Hkv"], 128)[at] = s["v"].double()[live]
        return tuple(out)
    dx, dw = [], []
    for n in "qk":
        # the chain rule through z = R (x w / norm), norm = sqrt(mean x^2 + eps)
        x, w, dz = s[n].double(), s["w" + n].double(), s["d%s_out" % n].double()
        dy = diag * dz + (off * dz)[..., partner]
        norm = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        dw.append((dy * x / norm).sum((0, 1, 2)))
        dnorm = -(dy * w * x).sum(-1, keepdim=True) / norm.pow(2)
        dx.append(dy * w / norm + dnorm * x / (norm * x.shape[-1]))
    return dx[0], dx[1], dw[0], dw[1]


def _exact_decode(s):
    B, Hq, Hkv, ps = s["B"], s["Hq"], s["Hkv"], s["page"]
    out = torch.zeros(B, Hq, 1, 128, device=DEV, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, device=DEV, dtype=torch.float64)
    group = {b: i for i in range(len(s["plens"])) for b in range(s["starts"][i], s["starts"][i + 1])}

    def rows(cache, table, n):
        return cache[table[: _ceil(n, ps)].long()].reshape(-1, Hkv, 128)[:n].double()

    shared = {}
    for b in range(B):
        i = group.get(b)
        if i is not None and i not in shared:
            shared = {i: [rows(s[c], s["prefix_table"][i], s["plens"][i]) for c in ("k_cache", "v_cache")]}
        n = s["own_lens"][b]
        k, v = (rows(s[c], s["block_table"][b], n) for c in ("k_cache", "v_cache"))
        if i is not None:
            k, v = torch.cat([shared[i][0], k]), torch.cat([shared[i][1], v])
        if len(k) == 0:
            continue
        q = s["q"][b, :, 0].double().view(Hkv, -1, 128)
        x = torch.einsum("hgd,khd->hgk", q, k) / math.sqrt(128)
        z = torch.logsumexp(x, -1)
        lse[b] = z.reshape(-1)
        out[b] = torch.einsum("hgk,khd->hgd", (x - z[..., None]).exp(), v).reshape(Hq, 1, 128)
    return out, lse
