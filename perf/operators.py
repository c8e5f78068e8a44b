"""Cases of the operators around the decode step: rotary positions, appending to a paged cache (bf16, or 8 bits with a
scale per page and KV head), decode attention over that cache, and causal attention over packed prompts.

``own`` False computes the plain forms with elementary torch operations in 32 bits; True calls the library.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100


# ------------------------------------------------------------------ the cases
def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128}
    return [
        # one decode step of 16 requests: q and k of the fused projection, latency only
        {"name": "rope_step_16", "op": "rope", "tokens": 16, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "banded", "base": 500000.0, "max_pos": 131072},
        # prompts of 16411 tokens in all: pairs side by side, half of the head, far positions
        {"name": "rope_prompt_partial", "op": "rope", "tokens": 16411, "hq": 32, "hkv": 8, "d": 128, "rot": 64,
         "interleaved": True, "scaling": "ramp", "base": 10000.0, "max_pos": 1048576},
        # one token for each of 64 requests into an 8-bit cache, pages partly filled
        {"name": "append_step_64_e4m3", "op": "append", **llama, "batch": 64, "tokens": 64, "page": 32, "bits": 8,
         "max_start": 2048, "rot": 128, "interleaved": False, "with_k": False},
        # four prompts (16391 tokens) behind short prefixes into an 8-bit cache; the rotated keys for the prompt attention
        {"name": "append_prompt_e4m3", "op": "append", **llama, "batch": 4, "tokens": 16391, "page": 64, "bits": 8,
         "max_start": 200, "rot": 128, "interleaved": False, "with_k": True},
        # ragged prompts into a bf16 cache of a small model
        {"name": "append_prompt_bf16", "op": "append", "hq": 8, "hkv": 2, "d": 64, "batch": 9, "tokens": 5003, "page": 16,
         "bits": 16, "max_start": 40, "rot": 32, "interleaved": True, "with_k": True},
        # one request of the small configuration: latency only
        {"name": "paged_1x4096_bf16", "op": "paged", "hq": 8, "hkv": 2, "d": 64, "batch": 1, "lo": 4096, "hi": 4096,
         "page": 16, "bits": 16, "blocks": 0},
        # the decode layer at 32K context, 16 requests
        {"name": "paged_16x32k_e4m3", "op": "paged", **llama, "batch": 16, "lo": 32768, "hi": 32768, "page": 32, "bits": 8,
         "blocks": 0},
        # long ragged contexts
        {"name": "paged_16x64k_128k_e4m3", "op": "paged", **llama, "batch": 16, "lo": 65536, "hi": 131072, "page": 64,
         "bits": 8, "blocks": 0},
        # 72 selected blocks for each KV head of a 64K context (sparse attention over the resident cache)
        {"name": "paged_selected_e4m3", "op": "paged", "hq": 64, "hkv": 8, "d": 128, "batch": 8, "lo": 65000, "hi": 65536,
         "page": 64, "bits": 8, "blocks": 72},
        # a ragged batch of short prompts, one of them a single token
        {"name": "prompt_ragged_short", "op": "prompt", "hq": 8, "hkv": 2, "d": 64, "batch": 13, "tokens": 2203, "past": 0},
        # one whole long prompt
        {"name": "prompt_16384", "op": "prompt", **llama, "batch": 1, "tokens": 16384, "past": 0},
        # prompts continued behind 6000 cached tokens each (a chunk of a longer prompt)
        {"name": "prompt_chunks", "op": "prompt", **llama, "batch": 3, "tokens": 4099, "past": 6000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "paged", "prompt"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    hq = hq if hq <= 64 else hkv * 4
    rot = rng.choice([d, d, d // 2])
    inter = rng.random() < 0.5
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 16411) if hq + hkv <= 40 else _log(rng, 1, 9000), "hq": hq, "hkv": hkv,
                "d": d, "rot": rot, "interleaved": inter, "scaling": rng.choice(["none", "linear", "banded", "ramp"]),
                "base": rng.choice([10000.0, 500000.0]), "max_pos": _log(rng, 100, 1048576)}
    if op == "append":
        batch = _log(rng, 1, 128)
        tokens = batch if rng.random() < 0.4 else batch + _log(rng, 1, 8000)
        return {"op": op, "hq": min(hq, 4 * hkv), "hkv": hkv, "d": d, "batch": batch, "tokens": tokens,
                "page": rng.choice([16, 32, 64, 128]), "bits": rng.choice([8, 8, 16]), "max_start": _log(rng, 1, 2000),
                "rot": rot, "interleaved": inter, "with_k": rng.random() < 0.5}
    if op == "paged":
        hi = _log(rng, 1, 131072)
        cap = max(1, (16 * 8 * 98304 * 128) // (hkv * d * max(hi, 1)))
        batch = min(_log(rng, 1, 128), cap)
        page = rng.choice([16, 32, 64, 128])
        bits = rng.choice([8, 8, 16])
        batch = max(1, batch // 2) if bits == 16 else batch
        blocks = _log(rng, 1, 128) if rng.random() < 0.35 and hi >= 128 * page else 0
        return {"op": op, "hq": hq, "hkv": hkv, "d": d, "batch": batch, "lo": max(1, hi // rng.choice([1, 2, 16])), "hi": hi,
                "page": page, "bits": bits, "blocks": blocks}
    batch = _log(rng, 1, 32)
    return {"op": op, "hq": min(hq, 32), "hkv": hkv, "d": d, "batch": batch, "tokens": batch + _log(rng, 1, 8000),
            "past": rng.choice([0, 0, _log(rng, 1, 2000)]) if batch <= 4 else 0}


# ------------------------------------------------------------------ inputs
def _spread(i):
    """A fixed ragged sequence in [0, 1)."""
    return (0.381966 + 0.618034 * i + 0.2 * ((i * i) % 5)) % 1.0


def _cuts(case):
    """Tokens of each packed request: at least one each, ragged, `tokens` in all."""
    b, t = case["batch"], case["tokens"]
    if t == b:
        return [1] * b
    weights = [_spread(i) ** 2 for i in range(b)]
    n = [1 + int((t - b) * w / sum(weights)) for w in weights]
    n[b // 2] += t - sum(n)
    return n


def _lens(case):
    """Context length of each request: the longest first, the others spread over the range."""
    lo, hi = case["lo"], case["hi"]
    return [hi] + [lo + int((hi + 1 - lo) * _spread(i)) for i in range(1, case["batch"])]


def _freq(rot, base=10000.0, scaling="none", factor=8.0, original=8192):
    """Turns per position of each pair in units of 2^-64, and the factor on the rotated values."""
    out, amp = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        wave = 2 * math.pi / f
        if scaling == "linear":
            f /= factor
        elif scaling == "banded":      # long waves slowed by the factor, short ones kept, a ramp between
            w = (original / wave - 1.0) / (4.0 - 1.0)
            w = min(1.0, max(0.0, w))
            f = (1 - w) * f / factor + w * f
        elif scaling == "ramp":        # the ramp runs over the pair's index instead
            lo = rot * math.log(original / (32 * 2 * math.pi)) / (2 * math.log(base))
            hi = rot * math.log(original / (1 * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = (1 - w) * f + w * f / factor
            amp = 0.1 * math.log(factor) + 1.0
        u = int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64
        out.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    return out, amp


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(g, *shape, channels=True):
    """bf16 values of projections: channels of unlike size, as keys have them."""
    x = torch.randn(*shape, generator=g, device="cuda")
    if channels:
        x = x * torch.exp(0.4 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x.bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t = case["tokens"]
        freq, s["amp"] = _freq(case["rot"], case["base"], case["scaling"])
        s["freq"] = torch.tensor(freq, dtype=torch.int64, device="cuda")
        s["qkv"] = _normal(g, t, hq + 2 * hkv, d)                # the fused projection; q and k are a view of it
        s["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda", dtype=torch.int32)
        return s
    if case["op"] == "prompt":
        n = _cuts(case)
        past = [0 if case["past"] == 0 else case["past"] + 7 * i for i in range(len(n))]
        cq, ck = [0], [0]
        for a, p in zip(n, past):
            cq.append(cq[-1] + a)
            ck.append(ck[-1] + a + p)
        s["cu_q"], s["cu_k"] = _i32(cq), _i32(ck)
        s["q"] = _normal(g, cq[-1], hq, d, channels=False)
        s["k"], s["v"] = _normal(g, ck[-1], hkv, d), _normal(g, ck[-1], hkv, d)
        return s
    page, b = case["page"], case["batch"]
    if case["op"] == "append":
        n = _cuts(case)
        start = torch.randint(0, case["max_start"], (b,), generator=g, device="cuda", dtype=torch.int32)
        need = (case["max_start"] + max(n) + page - 1) // page
        per = [(case["max_start"] + x + page - 1) // page for x in n]
        n_pages = sum(per) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(b, need, dtype=torch.int32, device="cuda")
        at = 0
        for i, p in enumerate(per):
            table[i, :p] = order[at:at + p]
            at += p
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        s["start"], s["table"] = start, table
        s["cu"] = None if case["tokens"] == b else _i32(cu)
        freq, s["amp"] = _freq(case["rot"])
        s["freq"] = torch.tensor(freq, dtype=torch.int64, device="cuda")
        s["q"], s["k"] = _normal(g, cu[-1], hq, d), _normal(g, cu[-1], hkv, d)
        s["v"] = _normal(g, cu[-1], hkv, d)
    else:
        lens = _i32(_lens(case))
        need = (case["hi"] + page - 1) // page
        n_pages = b * need
        s["table"] = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(b, need)
        s["lens"], s["max_len"] = lens, case["hi"]
        s["q"] = _normal(g, b, hq, d, channels=False)
        s["blocks"] = None
        if case["blocks"]:            # ascending distinct blocks of each KV head, the last one the newest
            k = case["blocks"]
            pick = torch.rand(b, hkv, need, generator=g, device="cuda")
            have = (lens + page - 1) // page
            at = torch.arange(need, device="cuda")
            pick = torch.where(at >= have[:, None, None], torch.zeros_like(pick), pick + (at == have[:, None, None] - 1))
            s["blocks"] = pick.topk(k, dim=-1).indices.sort(dim=-1).values.to(torch.int32).contiguous()
    shape = (n_pages, hkv, page, d)
    s["k_scale"] = s["v_scale"] = None
    if case["bits"] == 8:
        for x in ("k", "v"):
            codes = torch.empty(shape, dtype=E4M3, device="cuda")
            for i in range(0, n_pages, 4096):
                part = torch.randn(min(4096, n_pages - i), *shape[1:], generator=g, device="cuda")
                codes[i:i + 4096].copy_((part * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3))
            s[x + "_pages"] = codes
            s[x + "_scale"] = torch.ldexp(torch.ones(n_pages, hkv, device="cuda"),
                                              torch.randint(-8, -5, (n_pages, hkv), generator=g, device="cuda"))
    else:
        s["k_pages"], s["v_pages"] = _normal(g, *shape), _normal(g, *shape)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, freq, interleaved, amp, wide=False):
    """x [T][H][d] -> rotated, in 32 bits (64 where `wide`); the angle always in 64."""
    t = torch.float64 if wide else torch.float32
    n = freq.numel()
    turns = freq.double() / 2.0 ** 64
    turns = turns + (freq < 0)
    a = pos.double()[:, None] * turns
    a = (a - a.floor()) * (2 * math.pi)
    c, s = (a.cos() * amp).to(t)[:, None, :], (a.sin() * amp).to(t)[:, None, :]
    x = x.to(t)
    r = x[..., :2 * n]
    if interleaved:
        u, v = r[..., 0::2], r[..., 1::2]
        y = torch.stack((u * c - v * s, u * s + v * c), dim=-1).flatten(-2)
    else:
        u, v = r[..., :n], r[..., n:]
        y = torch.cat((u * c - v * s, u * s + v * c), dim=-1)
    return torch.cat((y, x[..., 2 * n:]), dim=-1)


def _places(s):
    """Request, position, page and row of every packed token."""
    table, start, t = s["table"], s["start"], s["k"].shape[0]
    at = torch.arange(t, device="cuda")
    cu = torch.arange(table.shape[0] + 1, device="cuda") if s["cu"] is None else s["cu"].long()
    req = torch.searchsorted(cu[1:], at, right=True)
    pos = start.long()[req] + at - cu[req]
    page = s["k_pages"].shape[2]
    return cu, pos, table[req, pos // page].long(), pos % page


def _pow2_scale(amax):
    m, e = torch.frexp(amax)
    e = torch.where(m <= E4M3_MAX / 512.0, e - 9, e - 8)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax)).clamp(min=SCALE_MIN)


def _store(pages, scale, x, s, cu, page_of, row):
    """Writes the bf16 rows x [T][Hkv][d] into their pages."""
    if scale is None:
        pages[page_of, :, row] = x
        return
    n_pages, hkv, page, d = pages.shape
    x = x.float()
    amax = torch.zeros(n_pages, hkv, device="cuda")
    amax.index_reduce_(0, page_of, x.abs().amax(-1), "amax")
    touched = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    touched[page_of] = True
    fresh = torch.zeros(n_pages, device="cuda").index_reduce_(0, page_of, (row == 0).float(), "amax").bool()
    new = _pow2_scale(amax)
    new = torch.where(fresh[:, None], new, torch.maximum(new, scale))
    new = torch.where(touched[:, None], new, scale)
    first = s["table"].gather(1, (s["start"].long() // page)[:, None])[:, 0].long()      # each request's first page
    keep = (s["start"].long() % page)[:, None] > torch.arange(page, device="cuda")       # rows that it has already
    keep = keep & (cu[1:] > cu[:-1])[:, None]
    raw = pages.view(torch.uint8)
    old = raw[first]
    again = (old.view(E4M3).float() * (scale / new)[first][:, :, None, None]).to(E4M3).view(torch.uint8)
    raw[first] = torch.where(keep[:, None, :, None], again, old)
    raw[page_of, :, row] = (x * (1.0 / new)[page_of][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(new)


def _plain_append(s):
    c = s["case"]
    cu, pos, page_of, row = _places(s)
    k = _rotate(s["k"], pos, s["freq"], c["interleaved"], s["amp"]).bfloat16()
    q = _rotate(s["q"], pos, s["freq"], c["interleaved"], s["amp"]).bfloat16()
    _store(s["k_pages"], s["k_scale"], k, s, cu, page_of, row)
    _store(s["v_pages"], s["v_scale"], s["v"], s, cu, page_of, row)
    return q, (k if c["with_k"] else None)


def _softmax(x):
    """In place: exp(x - max), and the log of the sum; a row of -inf gives zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    return total, m + total.log()


def _plain_paged(s):
    c = s["case"]
    page, r = c["page"], c["hq"] // c["hkv"]
    b, need = s["table"].shape
    hkv, d = c["hkv"], c["d"]
    heads = torch.arange(hkv, device="cuda")[None, :, None]
    if s["blocks"] is None:
        logical = torch.arange(need, device="cuda").expand(b, hkv, need)
    else:
        logical = s["blocks"].long()
    phys = s["table"].long()[:, None, :].expand(b, hkv, need).gather(2, logical)

    def rows(pages, scale):
        if scale is None:
            x = pages[phys, heads].float()
        else:
            x = pages.view(torch.uint8)[phys, heads].view(E4M3).float()
            x.mul_(scale[phys, heads][..., None, None])
        return x.flatten(2, 3)                                    # [b][Hkv][n][d]

    at = (logical[..., None] * page + torch.arange(page, device="cuda")).flatten(2)
    q = s["q"].float().view(b, hkv, r, d)
    x = torch.matmul(q, rows(s["k_pages"], s["k_scale"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    x.masked_fill_((at >= s["lens"][:, None, None])[:, :, None, :], -math.inf)
    total, lse = _softmax(x)
    o = torch.matmul(x, rows(s["v_pages"], s["v_scale"])) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(b, hkv * r, d).bfloat16(), lse.reshape(b, hkv * r)


def _plain_prompt(s):
    c = s["case"]
    r, d = c["hq"] // c["hkv"], c["d"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    iq, ik = torch.arange(s["q"].shape[0], device="cuda"), torch.arange(s["k"].shape[0], device="cuda")
    bq, bk = torch.searchsorted(cq[1:], iq, right=True), torch.searchsorted(ck[1:], ik, right=True)
    last = ck[bq + 1] - cq[bq + 1] + iq                           # the last key row that each query row sees
    hide = (bq[:, None] != bk[None, :]) | (ik[None, :] > last[:, None])
    k = s["k"].float().repeat_interleave(r, dim=1).permute(1, 2, 0)
    x = torch.matmul(s["q"].float().transpose(0, 1), k).mul_(1.0 / math.sqrt(d))
    x.masked_fill_(hide, -math.inf)
    total, lse = _softmax(x)
    o = torch.matmul(x, s["v"].float().repeat_interleave(r, dim=1).transpose(0, 1))
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o.transpose(0, 1).bfloat16(), lse[..., 0].t()


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from sparse_kv_cache_landmark_gb300 import kvo
        if op == "rope":
            return kvo.rope(s["qkv"][:, :c["hq"] + c["hkv"]], s["pos"], s["freq"], interleaved=c["interleaved"],
                            amplitude=s["amp"])
        if op == "append":
            k_out = torch.empty_like(s["k"]) if c["with_k"] else None
            q = kvo.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["start"], cu=s["cu"],
                                 k_scale=s["k_scale"], v_scale=s["v_scale"], freq=s["freq"],
                                 interleaved=c["interleaved"], amplitude=s["amp"], q=s["q"], k_out=k_out)
            return [q, k_out, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]]
        if op == "paged":
            return kvo.paged_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"], blocks=s["blocks"], max_len=s["max_len"])
        return kvo.prompt_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    if op == "rope":
        return _rotate(s["qkv"][:, :c["hq"] + c["hkv"]], s["pos"], s["freq"], c["interleaved"], s["amp"]).bfloat16()
    if op == "append":
        q, k_out = _plain_append(s)
        return [q, k_out, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]]
    if op == "paged":
        return _plain_paged(s)
    return _plain_prompt(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t, h = case["tokens"], hq + hkv
        return {"bytes": 4 * t * h * d + 4 * t + 4 * case["rot"], "flops": 3 * t * h * case["rot"]}
    if case["op"] == "append":
        t, w = case["tokens"], case["bits"] // 8
        kv = t * hkv * d
        scales = 0 if w == 2 else 2 * 4 * hkv * (t // case["page"] + case["batch"])
        return {"bytes": 4 * kv + 2 * w * kv + 4 * t * hq * d + (2 * kv if case["with_k"] else 0) + scales,
                "flops": 3 * t * (hq + hkv) * case["rot"] + (0 if w == 2 else 4 * kv)}
    if case["op"] == "paged":
        b, w = case["batch"], case["bits"] // 8
        most = case["blocks"] * case["page"] if case["blocks"] else case["hi"]
        mean = sum(min(n, most) for n in _lens(case)) / b
        n = b * hkv * mean
        scales = 0 if w == 2 else 2 * 4 * n / case["page"]
        return {"bytes": 2 * w * n * d + scales + 2 * b * hq * d * 2 + 4 * b * hq + 4 * n / case["page"] / hkv,
                "flops": 4 * b * hq * mean * d}
    n = _cuts(case)
    past = [0 if case["past"] == 0 else case["past"] + 7 * i for i in range(len(n))]
    pairs = sum(a * (a + 1) // 2 + a * p for a, p in zip(n, past))
    tk = sum(n) + sum(past)
    return {"bytes": 2 * d * (2 * sum(n) * hq + 2 * tk * hkv) + 4 * sum(n) * hq, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rotate(x, pos, freq, interleaved, amp):
    x = x.double()
    y = x.clone()
    n = len(freq)
    for i, f in enumerate(freq.tolist()):
        turn = (f % 2 ** 64) / 2 ** 64
        a = torch.remainder(pos.double() * turn, 1.0) * (2 * math.pi)
        c, s = amp * torch.cos(a)[:, None], amp * torch.sin(a)[:, None]
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., p] * s + x[..., q] * c
    return y


def _exact_attention(q, k, v, seen):
    """q [m][d], k and v [n][d], the first seen[i] keys for row i; all 64 bits."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    x = q @ k.t() / math.sqrt(q.shape[1])
    x = torch.where(torch.arange(k.shape[0], device="cuda")[None, :] < seen[:, None], x, -math.inf)
    lse = torch.logsumexp(x, dim=1)
    w = torch.where(torch.isinf(lse)[:, None], 0.0, torch.exp(x - lse[:, None]))
    return w @ v, lse


def _exact_append(c, s):
    page = c["page"]
    start, table = s["start"].tolist(), s["table"].tolist()
    cu = list(range(c["batch"] + 1)) if s["cu"] is None else s["cu"].tolist()
    pos = torch.cat([torch.arange(cu[b + 1] - cu[b], device="cuda") + start[b] for b in range(c["batch"])])
    q = _exact_rotate(s["q"], pos, s["freq"], c["interleaved"], s["amp"])
    k = _exact_rotate(s["k"], pos, s["freq"], c["interleaved"], s["amp"])
    out = [q, k if c["with_k"] else None]
    pages, scales = [], []
    for x, name in ((k.bfloat16().double(), "k"), (s["v"].double(), "v")):
        pool = s[name + "_pages"].double()
        scale = None if c["bits"] == 16 else s[name + "_scale"].double()
        for b in range(c["batch"]):
            at, end = start[b], start[b] + cu[b + 1] - cu[b]
            while at < end:
                lo, n = at % page, min(page - at % page, end - at)
                p = table[b][at // page]
                rows = x[cu[b] + at - start[b]: cu[b] + at - start[b] + n].transpose(0, 1)      # [Hkv][n][d]
                if scale is None:
                    pool[p, :, lo:lo + n] = rows
                else:
                    top = rows.abs().amax(dim=(1, 2))
                    size = torch.ldexp(torch.ones_like(top), torch.log2(top / E4M3_MAX).round().clamp(min=-99).int() - 1)
                    for _ in range(2):        # the smallest power of two that holds the largest value
                        size = torch.where(size * E4M3_MAX < top, 2 * size, size)
                    if lo:
                        size = torch.maximum(size, scale[p])
                        pool[p, :, :lo] *= (scale[p] / size)[:, None, None]
                    scale[p] = size
                    pool[p, :, lo:lo + n] = rows / size[:, None, None]
                at += n
        pages.append(pool)
        scales.append(scale)
    return out + pages + scales


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _exact_rotate(s["qkv"][:, :c["hq"] + c["hkv"]], s["pos"], s["freq"], c["interleaved"], s["amp"])
    if c["op"] == "append":
        return _exact_append(c, s)
    r, d = c["hq"] // c["hkv"], c["d"]
    if c["op"] == "paged":
        b, page = c["batch"], c["page"]
        o = torch.zeros(b, c["hq"], d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(b, c["hq"], dtype=torch.float64, device="cuda")
        lens = s["lens"].tolist()
        for i in range(b):
            for g in range(c["hkv"]):
                if s["blocks"] is None:
                    blocks = torch.arange((lens[i] + page - 1) // page, device="cuda")
                else:
                    blocks = s["blocks"][i, g].long()
                    blocks = blocks[blocks * page < lens[i]]
                n = int(((lens[i] - blocks * page).clamp(max=page)).sum())
                at = s["table"][i].long()[blocks]
                k, v = (s[x + "_pages"].view(torch.uint8 if c["bits"] == 8 else torch.bfloat16)[at, g] for x in "kv")
                if c["bits"] == 8:
                    k = k.view(E4M3).double() * s["k_scale"][at, g].double()[:, None, None]
                    v = v.view(E4M3).double() * s["v_scale"][at, g].double()[:, None, None]
                k, v = k.double().flatten(0, 1)[:n], v.double().flatten(0, 1)[:n]      # only the last block is short
                rows = slice(g * r, (g + 1) * r)
                o[i, rows], lse[i, rows] = _exact_attention(s["q"][i, rows].double(), k, v,
                                                            torch.full((r,), n, device="cuda"))
        return o, lse
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    o = torch.zeros(cq[-1], c["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(cq[-1], c["hq"], dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(c["hq"]):
            k = s["k"][ck[b]:ck[b + 1], h // r].double()
            v = s["v"][ck[b]:ck[b + 1], h // r].double()
            for i in range(0, nq, 4096):
                m = min(4096, nq - i)
                seen = nk - nq + i + 1 + torch.arange(m, device="cuda")
                top = nk - nq + i + m
                rows = slice(cq[b] + i, cq[b] + i + m)
                o[rows, h], lse[rows, h] = _exact_attention(s["q"][rows, h].double(), k[:top], v[:top], seen)
    return o, lse
