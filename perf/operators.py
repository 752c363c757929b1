"""Cases and plain forms of the attention operators: rotary positions, the
append to an 8-bit paged cache, attention over that cache, and the step that
runs the three on the packed rows of a projection.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU,
`run()` one pass (elementary torch operations, or this library's calls where
`own` is true), `work()` what a pass cannot do without and `exact()` the
results in 64 bits.
"""
import functools
import math
import random

import torch

own = False

NAN_CODE = 0x7F
MIN_EXP = -100          # the smallest block scale is 2^MIN_EXP
EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def _case(op, **kw):
    c = dict(op=op, q_heads=16, kv_heads=2, head_dim=128, page=64, rot=64, layout="half",
             scaling="plain", norm=False, window=0, seqs=1, ctx=0, new=1, ragged=False, far=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's q and k heads, a quarter of each head rotated after its norm
        dict(_case("rope", rot=32, norm=True, far=5000), name="rope_row"),
        # a long prompt's q and k heads at far positions, whole heads rotated, frequencies
        # scaled for a long context
        dict(_case("rope", q_heads=16, kv_heads=4, rot=128, layout="interleaved",
                   scaling="by_parts", new=16384, far=1000000), name="rope_prompt"),
        # one token of each of 64 sequences into the cache
        dict(_case("append", kv_heads=4, seqs=64, ctx=4000, ragged=True), name="append_step"),
        # three prompts of odd lengths into the cache at once
        dict(_case("append", kv_heads=4, seqs=3, new=7000, ctx=900, ragged=True),
             name="append_prompts"),
        # one decode step of one sequence: the latency case
        dict(_case("attention", ctx=4095), name="decode_row"),
        # one decode step of 64 sequences of different lengths: the bandwidth case
        dict(_case("attention", q_heads=32, kv_heads=4, seqs=64, ctx=16384, ragged=True),
             name="decode_batch"),
        # one decode step of one very long sequence: few rows, a long axis
        dict(_case("attention", q_heads=16, kv_heads=4, ctx=262143, page=128), name="decode_long"),
        # eight streams' frames of eleven rows each, three query heads to a key head
        dict(_case("attention", q_heads=24, kv_heads=8, head_dim=64, page=16, seqs=8, new=11,
                   ctx=1500), name="frames"),
        # a 1024-row prompt chunk after 7168 earlier tokens, wide heads
        dict(_case("attention", kv_heads=4, head_dim=256, page=32, ctx=7168, new=1024),
             name="prompt_chunk"),
        # a whole long prompt
        dict(_case("attention", page=128, new=16384), name="prompt"),
        # the whole attention step of one row, from the projection's packed row
        dict(_case("step", ctx=2047, norm=True), name="step_row"),
        # the whole attention step of a prompt chunk
        dict(_case("step", kv_heads=4, ctx=3000, new=1024, norm=True), name="step_chunk"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "step"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8] if kv > 1 else [4, 8, 16])
    d = rng.choice([64, 128, 128, 256])
    rot = rng.choice([d, d // 2, d // 4])
    c = _case(op, q_heads=kv * group, kv_heads=kv, head_dim=d, page=rng.choice([16, 32, 64, 128]),
              rot=rot, layout=rng.choice(["half", "interleaved"]),
              scaling=rng.choice(["plain", "linear", "by_parts"]), norm=rng.random() < 0.5,
              window=rng.choice([0, 0, _log(rng, 100, 5000)]))
    if op == "rope":
        c.update(new=min(_log(rng, 1, 16384), (16384 * 2560) // ((kv * group + kv) * d)),
                 far=_log(rng, 10, 2000000))
    elif op == "append":
        c.update(seqs=_log(rng, 1, 64), ragged=rng.random() < 0.7, ctx=_log(rng, 1, 4000))
        c["new"] = rng.choice([1, min(_log(rng, 2, 8000), 8192000 // (c["seqs"] * kv * d))])
    elif rng.random() < 0.5:      # single tokens
        c.update(seqs=_log(rng, 1, 64), ragged=rng.random() < 0.7, new=1)
        c["ctx"] = _log(rng, 1, min(200000, 400000000 // (c["seqs"] * kv * d)))
    else:                         # several rows of each sequence
        c.update(seqs=_log(rng, 1, 8), ragged=rng.random() < 0.7, new=_log(rng, 2, 4000),
                 ctx=_log(rng, 1, 8000))
        # at most the pairs of 16 heads over 8192 x 8192
        while c["seqs"] * c["new"] * (c["new"] + c["ctx"]) * c["q_heads"] > 16 * 8192 * 8192:
            c["new"] = max(2, c["new"] // 2)
            c["ctx"] = max(1, c["ctx"] * 3 // 4)
            c["seqs"] = max(1, c["seqs"] - 1)
    return c


def _lens(case):
    """(rows, cache length with the rows) of each sequence, from the case alone."""
    n = case["seqs"]
    if not case["ragged"]:
        return [case["new"]] * n, [case["ctx"] + case["new"]] * n
    r = random.Random(1000003 * n + 1009 * case["ctx"] + case["new"])
    rows = [max(1, int(case["new"] * r.uniform(0.3, 1.0))) for _ in range(n)]
    return rows, [k + int(case["ctx"] * r.uniform(0.1, 1.0)) for k in rows]


# ---- inputs -----------------------------------------------------------------

def _freqs(case):
    """Radians a position turns each pair by, in 64 bits; and the amplitude."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "by_parts":
        turns = 8192 * f / (2 * math.pi)
        g = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * (g + (1 - g) / 8.0), 1.2
    return f, 1.0


@functools.lru_cache(maxsize=8)
def _handle(q_heads, kv_heads, head_dim, page, rot, layout, scaling, window, rows, seqs):
    """The library's handle for a shape, which a serving program keeps for its life."""
    import block_fp8_mixture_router_gb300 as moe
    shape = moe.AttnShape(
        q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_tokens=page, rotary_dim=rot,
        rope_layout=layout, rope_base=10000.0, rope_scaling=scaling,
        rope_factor={"linear": 4.0, "by_parts": 8.0}.get(scaling, 1.0),
        rope_trained_positions=8192, rope_turns_low=1.0, rope_turns_high=32.0,
        rope_amplitude=1.2 if scaling == "by_parts" else 1.0, window=window)
    return moe.Attention(shape, max_rows=rows, max_seqs=seqs)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    n_rows, kv = _lens(case)
    rows = sum(n_rows)
    s = dict(case=case, rows=rows, max_rows=max(n_rows), max_kv=max(kv))
    freq, amp = _freqs(case)
    s["freq"], s["amp"] = freq.to(dev), amp
    if case["norm"]:
        s["q_gamma"] = (1 + 0.1 * randn(d)).to(torch.bfloat16)
        s["k_gamma"] = (1 + 0.1 * randn(d)).to(torch.bfloat16)
    else:
        s["q_gamma"] = s["k_gamma"] = None
    if case["op"] == "rope":
        # q and k heads side by side in one row; far positions in ascending order
        s["x"] = randn(rows, hq + hk, d).to(torch.bfloat16)
        first = torch.randint(0, case["far"], (1,), generator=g, device=dev)
        s["positions"] = (first + torch.arange(rows, device=dev)).to(torch.int32)
        s["out"] = torch.empty_like(s["x"])
    else:
        # the paged cache: shuffled pages, keys with a common direction per head
        # (as projections with a bias give), pages of unlike magnitude
        per = [-(-k // page) for k in kv]
        n_pages = sum(per) + 3
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        width = max(per)
        s["pages"] = torch.zeros((len(kv), width), dtype=torch.int32, device=dev)
        start = 0
        for i, n in enumerate(per):
            s["pages"][i, :n] = order[start:start + n]
            start += n
        begins = [0]
        for n in n_rows:
            begins.append(begins[-1] + n)
        s["row_start"] = torch.tensor(begins, dtype=torch.int32, device=dev)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        for name in ("k", "v"):
            big = torch.exp2(torch.round(0.5 * randn(n_pages, hk, 1, 1)))
            x = randn(n_pages, hk, page, d)
            if name == "k":
                x += randn(1, hk, 1, d)
            x *= big
            codes, scales = _quantise(x, x.abs().amax(dim=(2, 3)))
            s[name + "_codes"], s[name + "_scales"] = codes, scales
        if case["op"] == "append":
            s["k"] = randn(rows, hk, d).to(torch.bfloat16)
            s["v"] = randn(rows, hk, d).to(torch.bfloat16)
        elif case["op"] == "attention":
            s["q"] = randn(rows, hq, d).to(torch.bfloat16)
            s["out"] = torch.empty_like(s["q"])
        else:
            s["qkv"] = randn(rows, hq + 2 * hk, d).to(torch.bfloat16)
            s["out"] = torch.empty((rows, hq, d), dtype=torch.bfloat16, device=dev)
    if own:
        import block_fp8_mixture_router_gb300 as moe
        s["attn"] = _handle(hq, hk, d, page, case["rot"], case["layout"], case["scaling"],
                            case["window"], rows, case["seqs"])
        if case["op"] != "rope":
            s["cache"] = moe.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
            s["batch"] = moe.AttnBatch(s["row_start"], s["kv_len"], s["pages"], rows,
                                       max_seq_rows=s["max_rows"], max_kv_len=s["max_kv"])
    return s


# ---- plain forms ------------------------------------------------------------

def _quantise(x, amax):
    """x [pages, heads, tokens, D] in fp32 and each (page, head)'s largest magnitude ->
    e4m3 codes and the power-of-two scales."""
    m, e = torch.frexp(amax.float())
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, MIN_EXP)).clamp(min=MIN_EXP)
    scale = torch.ldexp(torch.ones_like(amax, dtype=torch.float32), k)
    codes = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def _rotate(x, positions, s):
    """Norm and rotation of x [rows, heads, D] (fp32); gamma by s["gamma"]."""
    case = s["case"]
    rot = case["rot"]
    turns = positions.double()[:, None] * (s["freq"] / (2 * math.pi))[None, :]
    turns = (turns - torch.round(turns)) * (2 * math.pi)
    cos = (torch.cos(turns) * s["amp"]).float()[:, None, :]
    sin = (torch.sin(turns) * s["amp"]).float()[:, None, :]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _norm(x, gamma):
    if gamma is None:
        return x
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * gamma.float()


def _places(s):
    """Sequence, position, page and slot of every row."""
    start, kv = s["row_start"].long(), s["kv_len"].long()
    row = torch.arange(s["rows"], device=start.device)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = kv[seq] - (start[seq + 1] - start[seq]) + (row - start[seq])
    page = s["pages"].long()[seq, pos // s["case"]["page"]]
    return seq, pos, page, pos % s["case"]["page"]


def _append(s, name, x):
    """x [rows, heads, D] bf16 into the cache's `name` pool."""
    codes, scales = s[name + "_codes"], s[name + "_scales"]
    page_tokens = s["case"]["page"]
    seq, pos, page, slot = _places(s)
    x = x.float()
    fine = torch.isfinite(x).all(dim=-1, keepdim=True)
    x = torch.where(fine, x, torch.zeros_like(x))
    amax = torch.zeros_like(scales)
    amax.scatter_reduce_(0, page[:, None].expand(-1, scales.shape[1]), x.abs().amax(dim=-1),
                         "amax")
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, MIN_EXP)).clamp(min=MIN_EXP)
    fresh = torch.ldexp(torch.ones_like(amax), k)
    # a page that earlier calls began: its scale only grows, its codes are rounded to it again
    n_rows = (s["row_start"][1:] - s["row_start"][:-1]).long()
    first = s["kv_len"].long() - n_rows
    begun = (first % page_tokens != 0) & (n_rows > 0)
    at = s["pages"].long()[torch.arange(len(first), device=first.device),
                           (first // page_tokens).clamp(max=s["pages"].shape[1] - 1)]
    old_scale = scales[at]
    grown = torch.where(begun[:, None], torch.maximum(fresh[at], old_scale), fresh[at])
    old = codes[at].view(torch.float8_e4m3fn).float() * (old_scale / grown)[:, :, None, None]
    kept = begun[:, None] & (torch.arange(page_tokens, device=at.device)[None, :]
                             < (first % page_tokens)[:, None])
    new = torch.where(kept[:, None, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8),
                      codes[at])
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=at.device)
    touched[page] = True
    at, grown, new = at[n_rows > 0], grown[n_rows > 0], new[n_rows > 0]
    scales.copy_(torch.where(touched[:, None], fresh, scales))
    scales[at] = grown
    codes[at] = new
    c = (x / scales[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    c = torch.where(fine, c, torch.full_like(c, NAN_CODE))
    codes[page, :, slot] = c


def _attend(s, q):
    """q [rows, heads, D] fp32 over the cache -> bf16."""
    case = s["case"]
    hk, d, page_tokens = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hk
    seq, pos, _, _ = _places(s)
    start, kv = s["row_start"].long(), s["kv_len"].long()
    n, most, longest = len(kv), s["max_rows"], s["max_kv"]
    j = torch.arange(longest, device=q.device)
    there = s["pages"].long()[:, j // page_tokens]                      # [seqs, keys]

    def values(name):
        c = s[name + "_codes"][there, :, j % page_tokens]               # [seqs, keys, heads, D]
        x = c.view(torch.float8_e4m3fn).float() * s[name + "_scales"][there][..., None]
        x = torch.where((j[None, :] < kv[:, None])[:, :, None, None], x, torch.zeros_like(x))
        return x.transpose(1, 2)                                        # [seqs, heads, keys, D]

    # rows of each sequence side by side, short ones padded
    r = torch.arange(most, device=q.device)
    at = (start[:-1, None] + r[None, :]).clamp(max=s["rows"] - 1)
    p = (kv - (start[1:] - start[:-1]))[:, None] + r[None, :]
    x = q[at].view(n, most, hk, group, d).permute(0, 2, 3, 1, 4).reshape(n, hk, group * most, d)
    w = torch.matmul(x, values("k").transpose(-1, -2)) * (1 / math.sqrt(d))
    w = w.view(n, hk, group, most, longest)
    sees = (j <= p[..., None]) & (j < kv[:, None, None])
    if case["window"]:
        sees &= j > p[..., None] - case["window"]
    w.masked_fill_(~sees[:, None, None], float("-inf"))
    top = w.amax(dim=-1, keepdim=True)
    w -= torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    w.exp_()
    z = w.sum(dim=-1, keepdim=True)
    o = torch.matmul(w.view(n, hk, group * most, longest), values("v"))
    o = o.view(n, hk, group, most, d) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, hk * group, d)
    return o[seq, torch.arange(s["rows"], device=q.device) - start[seq]].to(torch.bfloat16)


def _cache_outputs(s):
    return {n: s[n].view(torch.float8_e4m3fn) if n.endswith("codes") else s[n]
            for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def run(state):
    s, case = state, state["case"]
    hq, hk = case["q_heads"], case["kv_heads"]
    if own:
        attn = s["attn"]
        if case["op"] == "rope":
            return attn.rope(s["x"], s["positions"], gamma=s["q_gamma"], eps=EPS, out=s["out"])
        if case["op"] == "append":
            attn.append(s["k"], s["v"], s["cache"], s["batch"])
            return _cache_outputs(s)
        if case["op"] == "attention":
            return attn.forward(s["q"], s["cache"], s["batch"], out=s["out"])
        out = attn.step(s["qkv"], s["cache"], s["batch"], q_gamma=s["q_gamma"],
                        k_gamma=s["k_gamma"], eps=EPS, out=s["out"])
        return dict(_cache_outputs(s), out=out)
    if case["op"] == "rope":
        return _rotate(_norm(s["x"].float(), s["q_gamma"]), s["positions"], s).to(torch.bfloat16)
    if case["op"] == "append":
        _append(s, "k", s["k"])
        _append(s, "v", s["v"])
        return _cache_outputs(s)
    if case["op"] == "attention":
        return _attend(s, s["q"].float())
    pos = _places(s)[1]
    x = s["qkv"].float()
    q = _rotate(_norm(x[:, :hq], s["q_gamma"]), pos, s).to(torch.bfloat16)
    k = _rotate(_norm(x[:, hq:hq + hk], s["k_gamma"]), pos, s).to(torch.bfloat16)
    _append(s, "k", k)
    _append(s, "v", s["qkv"][:, hq + hk:])
    return dict(_cache_outputs(s), out=_attend(s, q.float()))


# ---- floors -----------------------------------------------------------------

def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    n_rows, kv = _lens(case)
    rows = sum(n_rows)
    if case["op"] == "rope":
        return {"bytes": 4 * rows * (hq + hk) * d + 4 * rows, "flops": 3 * rows * (hq + hk) * case["rot"]}
    new_pages = sum((k - 1) // case["page"] - (k - n) // case["page"] + 1 for n, k in zip(n_rows, kv))
    append = 2 * rows * hk * d * (2 + 1) + 2 * 4 * hk * new_pages
    if case["op"] == "append":
        return {"bytes": append, "flops": 2 * rows * hk * d}
    window = case["window"] or 1 << 60
    pairs = keys = 0
    for n, k in zip(n_rows, kv):
        first, last = k - n, k - 1                 # positions of the rows
        full = max(0, min(n, last - max(first, window - 1) + 1)) if window <= last else 0
        short = n - full                           # rows that see all earlier keys
        pairs += short * (first + 1) + short * (short - 1) // 2 + full * min(window, k)
        keys += min(k, window + n - 1)
    cache = keys * 2 * hk * (d + 4.0 / case["page"])
    flops = 4 * d * hq * pairs
    if case["op"] == "attention":
        return {"bytes": 4 * rows * hq * d + cache, "flops": flops}
    # the step reads the packed rows, writes its own part of the cache and reads the rest
    return {"bytes": 2 * rows * (2 * hq + 2 * hk) * d + append - 4 * rows * hk * d + cache
            - 2 * rows * hk * d, "flops": flops + 3 * rows * (hq + hk) * case["rot"]}


# ---- 64-bit results ---------------------------------------------------------

def _e4m3_values(device):
    """The finite non-negative e4m3 values in ascending order (code 0..126)."""
    c = torch.arange(127, device=device)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))


def _nearest_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, ties to the even code."""
    t = _e4m3_values(x.device)
    mid = (t[1:] + t[:-1]) / 2
    a = x.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    code = torch.where(lo == hi, lo, lo + lo % 2)   # on a midpoint: the even one of lo, lo + 1
    return torch.copysign(t[code], x)


def _exact_rope(case, s, x, gamma, positions):
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gamma.double()
    half = case["rot"] // 2
    pairs = torch.arange(half, device=x.device)
    one = pairs if case["layout"] == "half" else 2 * pairs
    two = one + (half if case["layout"] == "half" else 1)
    angle = torch.remainder(positions.double()[:, None] * s["freq"][None], 2 * math.pi)[:, None]
    turn = torch.polar(torch.full_like(angle, s["amp"]), angle)
    z = torch.complex(x[..., one], x[..., two]) * turn
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_append(case, s, name, x, n_rows, kv):
    """The pool's values / scale and scales after the append, page by page."""
    page = case["page"]
    val = s[name + "_codes"].view(torch.float8_e4m3fn).double()
    scales = s[name + "_scales"].double().clone()
    units, row = [], 0
    for i, (n, k) in enumerate(zip(n_rows, kv)):
        p = k - n
        while p < k:
            m = min(k, (p // page + 1) * page) - p
            units.append((i, p // page, p % page, row, m))
            p, row = p + m, row + m
    for u in units:
        i, pg, slot, row, m = u
        at = int(s["pages"][i, pg])
        new = x[row:row + m].double().transpose(0, 1)                  # [heads, m, D]
        top = new.abs().amax(dim=(1, 2))
        exp = torch.ceil(torch.log2(top / 448)).clamp(min=MIN_EXP)
        exp = torch.where(448 * torch.exp2(exp - 1) >= top, exp - 1, exp).clamp(min=MIN_EXP)
        sc = torch.exp2(exp)
        if slot:
            sc = torch.maximum(sc, scales[at])
            val[at, :, :slot] = _nearest_e4m3(val[at, :, :slot] * (scales[at] / sc)[:, None, None])
        val[at, :, slot:slot + m] = _nearest_e4m3(new / sc[:, None, None])
        scales[at] = sc
    return val, scales


def _exact_attention(case, s, q, kval, ksc, vval, vsc, n_rows, kv):
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hk
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    row = 0
    for i, (n, k) in enumerate(zip(n_rows, kv)):
        ids = s["pages"][i, :-(-k // page)].long()
        for h in range(hk):
            key = (kval[ids, h] * ksc[ids, h, None, None]).reshape(-1, d)[:k]
            val = (vval[ids, h] * vsc[ids, h, None, None]).reshape(-1, d)[:k]
            step = max(1, (1 << 28) // (group * k))
            for r in range(0, n, step):
                m = min(step, n - r)
                pos = torch.arange(k - n + r, k - n + r + m, device=q.device)
                low = max(0, k - n + r - case["window"] + 1) if case["window"] else 0
                high = k - n + r + m
                j = torch.arange(low, high, device=q.device)
                x = q[row + r:row + r + m, h * group:(h + 1) * group].double()
                w = torch.einsum("mgd,jd->gmj", x, key[low:high]) / math.sqrt(d)
                hide = j[None, :] > pos[:, None]
                if case["window"]:
                    hide |= j[None, :] <= pos[:, None] - case["window"]
                w = torch.softmax(w.masked_fill(hide[None], float("-inf")), dim=-1)
                out[row + r:row + r + m, h * group:(h + 1) * group] = torch.einsum(
                    "gmj,jd->mgd", w, val[low:high])
        row += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n_rows, kv = _lens(case)
    hq, hk = case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        return _exact_rope(case, s, s["x"], s["q_gamma"], s["positions"])

    def pool(name):
        return s[name + "_codes"].view(torch.float8_e4m3fn).double(), s[name + "_scales"].double()

    if case["op"] == "attention":
        return _exact_attention(case, s, s["q"], *pool("k"), *pool("v"), n_rows, kv)
    if case["op"] == "append":
        k, v = s["k"], s["v"]
    else:
        pos = torch.cat([torch.arange(b - a, b, device=s["qkv"].device) for a, b in zip(n_rows, kv)])
        x = s["qkv"]
        q = _exact_rope(case, s, x[:, :hq], s["q_gamma"], pos).to(torch.bfloat16)
        k = _exact_rope(case, s, x[:, hq:hq + hk], s["k_gamma"], pos).to(torch.bfloat16)
        v = x[:, hq + hk:]
    kval, ksc = _exact_append(case, s, "k", k, n_rows, kv)
    vval, vsc = _exact_append(case, s, "v", v, n_rows, kv)
    got = {"k_codes": kval, "k_scales": ksc, "v_codes": vval, "v_scales": vsc}
    if case["op"] == "step":
        got["out"] = _exact_attention(case, s, q, kval, ksc, vval, vsc, n_rows, kv)
    return got
