"""Workloads of the position rotation, the paged key/value cache and the attention over it.

Four operators, each in a plain form (elementary torch operations in 32 bits) and
as the calls a user makes of the framework (``own = True``):

  rope_fwd   per-head RMS norm of queries and keys and the position rotation,
             one pass (training and prompt processing)
  rope_bwd   its gradients (training)
  append     new tokens' queries normed and rotated, their keys normed, rotated
             and written, with the values, into a paged cache (serving)
  paged      attention of the new tokens over the paged cache (serving)

A case is a dict of plain values; ``prepare`` makes what a program holds before
the call, ``run`` is one pass, ``exact`` the definition in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(op, B, H, Hkv, L, d, dtype, layout, rotary, interleaved, norm=True, far=0):
    return dict(op=op, B=B, H=H, Hkv=Hkv, L=L, d=d, dtype=dtype, layout=layout, rotary=rotary,
                interleaved=interleaved, norm=norm, far=far)


def _paged(op, B, H, Hkv, d, dtype, n_lo, n_hi, len_lo, len_hi, page, layout, behind=0,
           rotary=0, interleaved=False, norm=False, causal=True):
    c = dict(op=op, B=B, H=H, Hkv=Hkv, d=d, dtype=dtype, n_lo=n_lo, n_hi=n_hi, len_lo=len_lo,
             len_hi=len_hi, page=page, layout=layout, behind=behind)
    if op == "append":
        c.update(rotary=rotary, interleaved=interleaved, norm=norm)
    else:
        c.update(causal=causal)
    return c


def listed():
    return [
        # a training step's forward on long sequences, between projections and attention
        dict(name="rope_fwd_train_b4_h16_l8192_d128",
             **_rope("rope_fwd", 4, 16, 16, 8192, 128, BF16, "bshd", 128, False)),
        # a short fp32 batch (parity runs, small models): launch latency
        dict(name="rope_fwd_f32_b2_h8_l32_d64",
             **_rope("rope_fwd", 2, 8, 8, 32, 64, F32, "bhsd", 64, True)),
        # the training step's backward with grouped key/value heads
        dict(name="rope_bwd_train_b2_h32_kv8_l4096_d128",
             **_rope("rope_bwd", 2, 32, 8, 4096, 128, BF16, "bshd", 128, False)),
        # decoder training on sentences, half of each head rotated, odd length
        dict(name="rope_bwd_dec_b128_h8_l127_d64",
             **_rope("rope_bwd", 128, 8, 8, 127, 64, BF16, "bhsd", 32, True)),
        # one generation step of 256 sentences: a token each into its page
        dict(name="append_step_b256_h8_d64",
             **_paged("append", 256, 8, 8, 64, BF16, 1, 1, 128, 1024, 16, "bshd", rotary=64,
                      norm=False)),
        # prompts of up to 2048 tokens written behind what is cached
        dict(name="append_prompt_b8_h32_kv8_d128",
             **_paged("append", 8, 32, 8, 128, BF16, 513, 2048, 1024, 4096, 64, "bhsd", behind=37,
                      rotary=128, norm=True)),
        # one user, one token, a short dialogue: latency
        dict(name="paged_one_h8_d64",
             **_paged("paged", 1, 8, 8, 64, BF16, 1, 1, 300, 300, 16, "bshd")),
        # one generation step of 256 sentences, small pages
        dict(name="paged_step_b256_h8_d64",
             **_paged("paged", 256, 8, 8, 64, BF16, 1, 1, 128, 1024, 16, "bshd")),
        # one generation step over long caches, grouped key/value heads
        dict(name="paged_step_b64_h32_kv8_d128",
             **_paged("paged", 64, 32, 8, 128, BF16, 1, 1, 4096, 8192, 64, "bshd")),
        # a serving batch of prompt chunks and single tokens together
        dict(name="paged_chunks_b8_h32_kv8_d128",
             **_paged("paged", 8, 32, 8, 128, BF16, 1, 512, 1000, 4096, 64, "bhsd", behind=19)),
        # a whole long prompt through the cache
        dict(name="paged_prompt_b1_h16_l8192_d128",
             **_paged("paged", 1, 16, 16, 128, BF16, 8192, 8192, 8192, 8192, 128, "bshd")),
        # a few drafted tokens of each sequence, fp32
        dict(name="paged_draft_f32_b8_h8_kv2_d64",
             **_paged("paged", 8, 8, 2, 64, F32, 5, 5, 90, 700, 32, "bshd")),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "append", "paged", "paged", "paged"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    while Hkv * group > 32:
        group = rng.choice([1, 2])
    H = Hkv * group
    layout = rng.choice(["bshd", "bhsd"])
    rotary = rng.choice([d, d, d // 2])
    inter = rng.random() < 0.5
    if op in ("rope_fwd", "rope_bwd"):
        B = _log_int(rng, 1, 128)
        L = _log_int(rng, 1, 8192)
        while B * L * (H + Hkv) * d * (2 if dtype == F32 else 1) > 1 << 27:
            L = max(1, L // 2) if L > B else L
            B = max(1, B // 2) if B > 1 else B
        return _rope(op, B, H, Hkv, L, d, dtype, layout, rotary, inter, norm=rng.random() < 0.7,
                     far=rng.choice([0, 0, 100000]))
    B = _log_int(rng, 1, 128)
    len_hi = _log_int(rng, 1, 8192)
    len_lo = rng.randint(max(1, len_hi // 4), len_hi)
    single = rng.random() < 0.5
    n_hi = 1 if single else min(len_lo, _log_int(rng, 2, 2048))
    n_lo = 1 if single else rng.randint(1, n_hi)
    most = 1 << 28 if dtype == BF16 else 1 << 26
    while B > 1 and (B * len_hi * Hkv * d > most or
                     B * n_hi * len_hi * H * d > (1 << 37 if dtype == BF16 else 1 << 33)):
        B //= 2
    while n_hi > 1 and B * n_hi * len_hi * H * d > (1 << 37 if dtype == BF16 else 1 << 33):
        n_hi = max(1, n_hi // 2)
        n_lo = min(n_lo, n_hi)
    page = rng.choice([16, 32, 64, 128, 256])
    behind = rng.choice([0, 0, rng.randint(1, 64)])
    if op == "append":
        return _paged(op, B, H, Hkv, d, dtype, n_lo, n_hi, len_lo, len_hi, page, layout, behind,
                      rotary, inter, rng.random() < 0.5)
    return _paged(op, B, H, Hkv, d, dtype, n_lo, n_hi, len_lo, len_hi, page, layout, behind,
                  causal=rng.random() < 0.85)


def _spread(lo, hi, B):
    return [lo + (hi - lo) * b // max(1, B - 1) if B > 1 else hi for b in range(B)]


def _lens(case):
    """New tokens and cached length (these tokens among them) of each sequence,
    the same for every seed but for their order: evenly spread over the ranges,
    the longest chunks behind the shortest caches."""
    n = _spread(case["n_lo"], case["n_hi"], case["B"])
    ln = _spread(case["len_lo"], case["len_hi"], case["B"])[::-1]
    return [(min(a, b), b) for a, b in zip(n, ln)]


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        rows = case["B"] * case["L"] * (H + Hkv)
        passes = 2 if case["op"] == "rope_fwd" else 3
        return {"bytes": passes * rows * d * e + 4 * case["B"] * case["L"],
                "flops": (10 if case["op"] == "rope_fwd" else 20) * rows * d}
    lens = _lens(case)
    T = sum(n for n, _ in lens)
    table = 4 * sum(-(-ln // case["page"]) for _, ln in lens)
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * Hkv) * d * e + 4 * T, "flops": 10 * T * (H + Hkv) * d}
    pairs = sum(n * ln - (n * (n - 1) // 2 if case["causal"] else 0) for n, ln in lens)
    return {"bytes": 2 * T * H * d * e + sum(ln for _, ln in lens) * Hkv * 2 * d * e + table,
            "flops": 4 * H * d * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _inv_freq(rotary):
    i = torch.arange(rotary // 2, dtype=torch.float64)
    return (BASE ** (-2.0 * i / rotary)).float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dt(case)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]

    def normal(*shape, amp=1.0, about=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * amp + about).to(dt)

    s = dict(case=case)
    if case.get("rotary"):
        s["inv_freq"] = _inv_freq(case["rotary"])
        # learned scales near one
        s["qw"] = normal(d, amp=0.1, about=1.0) if case["norm"] else None
        s["kw"] = normal(d, amp=0.1, about=1.0) if case["norm"] else None
    if case["op"] in ("rope_fwd", "rope_bwd"):
        B, L = case["B"], case["L"]
        shape = (lambda h: (B, L, h, d)) if case["layout"] == "bshd" else (lambda h: (B, h, L, d))
        s["q"], s["k"] = normal(*shape(H)), normal(*shape(Hkv))
        # positions of packed or shifted sequences
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(L, device="cuda")).to(torch.int32)
        if case["op"] == "rope_fwd":
            s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        else:
            s["gq"], s["gk"] = normal(*shape(H)), normal(*shape(Hkv))
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            s["dqw"] = torch.zeros(d, device="cuda") if case["norm"] else None
            s["dkw"] = torch.zeros(d, device="cuda") if case["norm"] else None
            if own:
                from transformer_head_scaled_mha_gb300 import mha_qk_norm_rope_bwd_workspace_size
                s["ws"] = torch.empty(mha_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8,
                                      device="cuda")
        return s
    # ragged sequences, in an order of their own, and pages taken from a pool in no order
    lens = _lens(case)
    B, page = case["B"], case["page"]
    order = torch.randperm(B, generator=g, device="cuda").cpu().tolist()
    lens = [lens[i] for i in order]
    T = sum(n for n, _ in lens)
    max_pages = -(-max(ln for _, ln in lens) // page) + 1
    used = sum(-(-ln // page) for _, ln in lens)
    pool = used + 3
    ids = torch.randperm(pool, generator=g, device="cuda")[:used].to(torch.int32).cpu()
    table = torch.zeros(B, max_pages, dtype=torch.int32)
    at = 0
    for b, (_, ln) in enumerate(lens):
        m = -(-ln // page)
        table[b, :m] = ids[at:at + m]
        at += m
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["table"] = table.cuda()
    s["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
    s["kvlen"] = torch.tensor([ln for _, ln in lens], dtype=torch.int32).cuda()
    s["max_q"], s["max_k"] = max(n for n, _ in lens), max(ln for _, ln in lens)
    rows = T + case["behind"]  # rows behind the last sequence, as a captured batch has them
    shape = (pool, page, Hkv, d) if case["layout"] == "bshd" else (pool, Hkv, page, d)
    s["kc"], s["vc"] = normal(*shape), normal(*shape)
    s["q"] = normal(rows, H, d)
    if case["op"] == "append":
        s["k"], s["v"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
        s["qo"] = torch.zeros_like(s["q"])
        return s
    s["out"] = torch.zeros_like(s["q"])
    s["scale"] = d ** -0.5
    if own:
        from transformer_head_scaled_mha_gb300 import mha_paged_workspace_size
        s["ws"] = torch.empty(mha_paged_workspace_size(B, rows, H, Hkv, d, s["max_q"], s["q"].dtype),
                              dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    import transformer_head_scaled_mha_gb300 as mha
    c = s["case"]
    if c["op"] == "rope_fwd":
        qo, ko = mha.mha_qk_norm_rope_fwd(
            s["q"], s["k"], s["qo"], s["ko"], q_weight=s["qw"], k_weight=s["kw"],
            positions=s["pos"], inv_freq=s["inv_freq"], layout=c["layout"],
            interleaved=c["interleaved"], eps=EPS)
        return {"q": qo, "k": ko}
    if c["op"] == "rope_bwd":
        dq, dk, dqw, dkw = mha.mha_qk_norm_rope_bwd(
            s["q"], s["k"], s["gq"], s["gk"], s["dq"], s["dk"], s["dqw"], s["dkw"],
            q_weight=s["qw"], k_weight=s["kw"], positions=s["pos"], inv_freq=s["inv_freq"],
            layout=c["layout"], interleaved=c["interleaved"], eps=EPS, workspace=s["ws"])
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    if c["op"] == "append":
        qo = mha.mha_paged_append(
            s["q"], s["k"], s["v"], s["kc"], s["vc"], s["qo"], q_starts=s["starts"],
            kv_lengths=s["kvlen"], block_table=s["table"], q_weight=s["qw"], k_weight=s["kw"],
            inv_freq=s["inv_freq"], layout=c["layout"], interleaved=c["interleaved"], eps=EPS)
        return {"q": qo, "k_cache": s["kc"], "v_cache": s["vc"]}
    out = mha.mha_paged_fwd(
        s["q"], s["kc"], s["vc"], s["out"], q_starts=s["starts"], kv_lengths=s["kvlen"],
        block_table=s["table"], max_q=s["max_q"], layout=c["layout"],
        mask_kind=mha.MHA_MASK_CAUSAL_TAIL if c["causal"] else mha.MHA_MASK_NONE,
        scale=s["scale"], workspace=s["ws"])
    return {"out": out}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _cos_sin(pos, inv_freq):
    """pos [...] -> cos, sin [..., rotary / 2]; the angle in 64 bits (far positions)."""
    a = pos.double()[..., None] * inv_freq.double()
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, interleaved, sign=1.0):
    """x [..., d] in 32 bits; the first 2 * cos.shape[-1] dimensions are rotated."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    sin = sin * sign
    u, v = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((u, v), dim=-1).flatten(-2) if interleaved else torch.cat((u, v), dim=-1)
    return torch.cat((rot, x[..., r:]), dim=-1)


def _norm_rope(x, w, cos, sin, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, cos, sin, interleaved).to(x.dtype)


def _norm_rope_bwd(x, w, dy, cos, sin, interleaved):
    g = _rotate(dy.float(), cos, sin, interleaved, sign=-1.0)
    if w is None:
        return g.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    n = x32 * r
    gw = g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * n).double().flatten(0, -2).sum(0).float()


def _head_axis(case):
    return 2 if case["layout"] == "bshd" else 1


def _tokens(s):
    """Sequence, index within it, position and validity of each row of q."""
    starts, kvlen = s["starts"].long(), s["kvlen"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = (torch.searchsorted(starts, t, right=True) - 1).clamp(0, len(kvlen) - 1)
    n = starts[1:] - starts[:-1]
    i = t - starts[seq]
    return seq, i, kvlen[seq] - n[seq] + i, t < starts[-1]


def _cache_rows(case, cache):
    """The cache as [pages, page, heads, d], whatever its layout."""
    return cache if case["layout"] == "bshd" else cache.transpose(1, 2)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] in ("rope_fwd", "rope_bwd"):
        cos, sin = (t.unsqueeze(_head_axis(c)) for t in _cos_sin(s["pos"], s["inv_freq"]))
        inter = c["interleaved"]
        if c["op"] == "rope_fwd":
            return {"q": _norm_rope(s["q"], s["qw"], cos, sin, inter),
                    "k": _norm_rope(s["k"], s["kw"], cos, sin, inter)}
        dq, dqw = _norm_rope_bwd(s["q"], s["qw"], s["gq"], cos, sin, inter)
        dk, dkw = _norm_rope_bwd(s["k"], s["kw"], s["gk"], cos, sin, inter)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    page = c["page"]
    seq, i, pos, valid = _tokens(s)
    if c["op"] == "append":
        cos, sin = (t[:, None] for t in _cos_sin(pos, s["inv_freq"]))
        q = torch.where(valid[:, None, None],
                        _norm_rope(s["q"], s["qw"], cos, sin, c["interleaved"]), s["qo"])
        k = _norm_rope(s["k"], s["kw"], cos, sin, c["interleaved"])
        # the rows behind the last sequence repeat the last token's write
        T = s["k"].shape[0] - c["behind"]
        row = torch.arange(s["k"].shape[0], device="cuda").clamp(max=T - 1)
        p = pos[row]
        slot = s["table"].long()[seq[row], p // page], p % page
        _cache_rows(c, s["kc"])[slot] = k[row]
        _cache_rows(c, s["vc"])[slot] = s["v"][row]
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    # every sequence's queries and keys side by side, padded to the longest
    starts, kvlen = s["starts"].long(), s["kvlen"].long()
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    j = torch.arange(s["max_k"], device="cuda")
    slot = s["table"].long()[:, j // page], (j % page)[None, :]
    live = j[None, :] < kvlen[:, None]
    K = _cache_rows(c, s["kc"])[slot].float()
    V = torch.where(live[:, :, None, None], _cache_rows(c, s["vc"])[slot].float(), 0.0)
    row = (starts[:-1, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=len(s["q"]) - 1)
    q = s["q"][row].float().unflatten(2, (Hkv, H // Hkv))
    sc = torch.einsum("bnghd,bkgd->bghnk", q, K) * s["scale"]
    n = (starts[1:] - starts[:-1])[:, None]
    last = kvlen[:, None] - n + torch.arange(s["max_q"], device="cuda") if c["causal"] else \
        (kvlen[:, None] - 1).expand(-1, s["max_q"])
    allowed = (j <= last[:, :, None]) & live[:, None, :]
    sc = sc.masked_fill(~allowed[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    w = (sc - torch.where(top == -math.inf, 0.0, top)).exp()
    o = torch.einsum("bghnk,bkgd->bnghd", w, V)
    total = w.sum(-1).permute(0, 3, 1, 2)[..., None]
    o = torch.where(total > 0, o / total, 0.0).flatten(2, 3)
    o = o[seq, i.clamp(0, s["max_q"] - 1)].to(s["q"].dtype)
    return {"out": torch.where(valid[:, None, None], o, s["out"])}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _define(x, w, pos, inv_freq, rotary, interleaved):
    """Norm, then each pair as a complex number times e^(i pos f); x [..., d] and
    pos in x's leading shape, 64 bits."""
    if w is not None:
        x = w * x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       pos[..., None] * inv_freq)
    z, rest = x[..., :rotary], x[..., rotary:]
    z = z.unflatten(-1, (rotary // 2, 2)) if interleaved else \
        z.unflatten(-1, (2, rotary // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, rest), -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    to64 = lambda t: None if t is None else t.double()  # noqa: E731
    if c["op"] in ("rope_fwd", "rope_bwd"):
        pos = s["pos"].double().unsqueeze(_head_axis(c))
        args = (to64(s["inv_freq"]), c["rotary"], c["interleaved"])
        if c["op"] == "rope_fwd":
            return {"q": _define(to64(s["q"]), to64(s["qw"]), pos, *args),
                    "k": _define(to64(s["k"]), to64(s["kw"]), pos, *args)}
        res = {}
        for x, w, g, a, b in (("q", "qw", "gq", "dq", "dqw"), ("k", "kw", "gk", "dk", "dkw")):
            leaf = to64(s[x]).requires_grad_()
            weight = to64(s[w])
            if weight is not None:
                weight.requires_grad_()
            _define(leaf, weight, pos, *args).backward(to64(s[g]))
            res[a], res[b] = leaf.grad, weight.grad if weight is not None else None
        return res
    starts, kvlen, table = (s[x].cpu().tolist() for x in ("starts", "kvlen", "table"))
    page = c["page"]
    if c["op"] == "append":
        q, kc, vc = to64(s["qo"]), to64(s["kc"]), to64(s["vc"])
        for b, ln in enumerate(kvlen):
            lo, hi = starts[b], starts[b + 1]
            pos = torch.arange(ln - (hi - lo), ln, device="cuda")
            args = (pos.double()[:, None], to64(s["inv_freq"]), c["rotary"], c["interleaved"])
            q[lo:hi] = _define(to64(s["q"][lo:hi]), to64(s["qw"]), *args)
            k = _define(to64(s["k"][lo:hi]), to64(s["kw"]), *args)
            where = s["table"][b][pos // page].long() * page + pos % page
            for cache, new in ((kc, k), (vc, to64(s["v"][lo:hi]))):
                if c["layout"] == "bshd":
                    cache.view(-1, c["Hkv"], c["d"])[where] = new
                else:
                    for h in range(c["Hkv"]):
                        cache[where // page, h, where % page] = new[:, h]
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if work(c)["flops"] > 4e12:
        return None
    out = to64(s["out"])
    for b, ln in enumerate(kvlen):
        lo, hi = starts[b], starts[b + 1]
        n = hi - lo
        ids = table[b][:-(-ln // page)]
        K, V = (torch.cat([cache[i] if c["layout"] == "bshd" else cache[i].transpose(0, 1)
                           for i in ids])[:ln] for cache in (s["kc"], s["vc"]))
        future = torch.ones(n, ln, dtype=torch.bool, device="cuda").triu(ln - n + 1) \
            if c["causal"] else None
        for h in range(c["H"]):
            kv = h // (c["H"] // c["Hkv"])
            logits = s["scale"] * (to64(s["q"][lo:hi, h]) @ to64(K[:, kv]).T)
            if future is not None:
                logits[future] = -math.inf
            out[lo:hi, h] = torch.softmax(logits, -1) @ to64(V[:, kv])
    return {"out": out}
