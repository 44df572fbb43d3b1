"""Measured cases of the paged key/value cache: appending to it (with the rotary rotation of keys and
queries on the way) and attention that reads it, in bf16 and in e4m3 with one scale for each page and
head.

A batch is ragged: sequence b has q_len(b) new tokens (rows cu_q[b] .. cu_q[b+1] of the token-major
tensors) and seq_lens[b] tokens in all, the new ones last; block_table[b] names its pages.  The plain
forms are elementary torch operations in 32 bits over the padded batch.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN_EXP = -100  # a page of zeros gets the scale 2^-100
ROPE_BASE = 10000.0


def _case(name, op, cache, B, Hq, Hkv, d, page, q_lo, q_hi, len_lo, len_hi, **more):
    c = {"name": name, "op": op, "cache": cache, "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page,
         "q_lo": q_lo, "q_hi": q_hi, "len_lo": len_lo, "len_hi": len_hi}
    c.update(more)
    return c


def listed():
    return [
        # one sequence generating: the smallest append of a serving loop, where latency is all
        _case("append one token bf16", "append", "bf16", 1, 32, 8, 128, 16, 1, 1, 500, 1000, rot=128, interleaved=False),
        # a decode batch of a continuous-batching server, ragged lengths, one token each
        _case("append batch e4m3", "append", "e4m3", 128, 32, 8, 128, 64, 1, 1, 100, 8000, rot=128, interleaved=False),
        # prompts of odd lengths, the first chunk of each, rotation over half of the head dimension in pairs
        _case("append prompts bf16", "append", "bf16", 7, 16, 4, 64, 32, 150, 1200, 150, 2500, rot=32, interleaved=True),
        # a large prefill chunk into the 8-bit cache
        _case("append prompts e4m3", "append", "e4m3", 4, 32, 8, 128, 16, 2000, 8192, 2000, 20000, rot=128, interleaved=False),
        # one user, short history: a chat's first answers
        _case("decode one short bf16", "attend", "bf16", 1, 32, 8, 128, 16, 1, 1, 300, 700),
        # a long document read by one user: few rows, a long axis
        _case("decode one long e4m3", "attend", "e4m3", 1, 32, 8, 128, 64, 1, 1, 120000, 131072),
        # a server's decode batch with ragged lengths
        _case("decode batch e4m3", "attend", "e4m3", 64, 32, 8, 128, 64, 1, 1, 200, 8192),
        # one key/value head per query head, small heads
        _case("decode batch mha bf16", "attend", "bf16", 32, 16, 16, 64, 32, 1, 1, 1000, 4096),
        # a few drafted tokens per sequence verified at once
        _case("verify drafts e4m3", "attend", "e4m3", 24, 32, 8, 128, 32, 3, 6, 1000, 6000),
        # a prompt chunk over the earlier chunks' cache
        _case("prefill chunk bf16", "attend", "bf16", 1, 32, 8, 128, 64, 2048, 2048, 16384, 16384),
        # several prompts of odd lengths in the 8-bit cache
        _case("prefill ragged e4m3", "attend", "e4m3", 4, 32, 8, 128, 16, 300, 1500, 1500, 8192),
        # prompt chunks and single tokens in one batch
        _case("mixed batch e4m3", "attend", "e4m3", 16, 16, 2, 128, 64, 1, 500, 600, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend"))
    cache = rng.choice(("bf16", "e4m3"))
    d = rng.choice((64, 128, 128))
    page = rng.choice((16, 32, 64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8))
    kind = rng.choice(("token", "token", "few", "chunk", "mixed"))
    while True:
        B = _log(rng, 1, 128 if kind == "token" else 32 if kind == "few" else 6)
        q_hi = 1 if kind == "token" else rng.randint(2, 9) if kind == "few" else _log(rng, 30, 2000)
        q_lo = 1 if kind != "chunk" else max(1, q_hi // rng.randint(1, 4))
        len_hi = max(q_hi + 1, _log(rng, 40, 60000 if op == "attend" else 20000))
        len_lo = max(1, len_hi // rng.randint(1, 20))
        c = _case("", op, cache, B, Hkv * G, Hkv, d, page, q_lo, q_hi, len_lo, len_hi)
        del c["name"]
        # no more than the largest listed ones: elements of the padded cache and of the padded scores
        if B * Hkv * len_hi * d <= 2 ** 29 and B * Hkv * G * q_hi * len_hi <= 2 ** 29:
            break
    if op == "append":
        c["rot"] = rng.choice((d, d, d // 2, 16))
        c["interleaved"] = rng.random() < 0.3
    return c


def _lengths(case):
    """New tokens and whole length of each sequence: spread evenly over the case's ranges, the same for every seed."""
    rng = np.random.default_rng([case[x] for x in ("B", "Hq", "Hkv", "d", "page", "q_hi", "len_hi")])
    q = rng.integers(case["q_lo"], case["q_hi"] + 1, case["B"])
    n = np.maximum(rng.integers(case["len_lo"], case["len_hi"] + 1, case["B"]), q)
    return q, n


def _needed_scale(amax):
    """The smallest power of two 2^e, e >= -100, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_MIN_EXP)).clamp(min=SCALE_MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantised_pages(x):
    """e4m3 pages and their scales [pages, heads] of values [pages, heads, page, d]."""
    s = _needed_scale(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, d, page = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    q_len, seq = _lengths(case)
    T = int(q_len.sum())
    used = -(-seq // page)
    max_pages = -(-case["len_hi"] // page)
    max_pages = max(max_pages, int(used.max()))
    n_pages = int(used.sum()) + 5
    # pages are handed out in no order, as a pool that has been in use for a while does
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(used)[:-1]])
    at = first[:, None] + np.minimum(np.arange(max_pages)[None, :], used[:, None] - 1)
    table = order[torch.from_numpy(at).to(dev)].contiguous()

    def pages(spread):
        # keys and values of differing size from page to page
        size = torch.exp2(torch.randn(n_pages, Hkv, 1, 1, generator=g, device=dev) * spread)
        x = torch.empty(n_pages, Hkv, page, d, dtype=torch.float32, device=dev).normal_(generator=g)
        x = x.mul_(size)
        return _quantised_pages(x) if case["cache"] == "e4m3" else (x.to(torch.bfloat16), None)

    k_pages, k_scale = pages(0.3)
    v_pages, v_scale = pages(0.5)

    def rows(heads):
        return torch.randn(T, heads, d, generator=g, device=dev).to(torch.bfloat16)

    s = {
        "case": case,
        "k_pages": k_pages, "v_pages": v_pages, "k_scale": k_scale, "v_scale": v_scale,
        "block_table": table,
        "cu_q": torch.from_numpy(np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)).to(dev),
        "seq_lens": torch.from_numpy(seq.astype(np.int32)).to(dev),
        "max_q": int(q_len.max()),
        "q": rows(Hq),
    }
    if case["op"] == "append":
        # keys and values are slices of one projection, as a model's fused product leaves them
        kv = rows(2 * Hkv)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        half = case["rot"] // 2
        freq = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(max_pages * page, dtype=torch.float64, device=dev)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        from exact_attention_159_b200 import api
        s["cache"] = api.PagedCache(k_pages, v_pages, k_scale, v_scale)
        s["batch"] = api.PagedBatch(s["block_table"], s["cu_q"], s["seq_lens"], s["max_q"])
    return s


def _where(s, T):
    """Sequence and position of each token row."""
    row = torch.arange(T, device=s["cu_q"].device)
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu, row, right=True) - 1
    return b, s["seq_lens"].long()[b] - cu[b + 1] + row


def _rotated(x, pos, cos, sin, rot, interleaved):
    x = x.float()
    c, n = cos[pos][:, None, :], sin[pos][:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * n, b * c + a * n), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _append_e4m3(pages, scale, x, page_of, off):
    """New values x [T, heads, d] into their slots; a page's scale grows to what they need, and the codes
    of the slots before the first of them with it."""
    n_pages, heads, size, d = pages.shape
    need = torch.zeros(n_pages, heads, device=x.device)
    need.index_reduce_(0, page_of, x.abs().amax(dim=2), "amax")
    need = _needed_scale(need)
    held = torch.full((n_pages,), size, device=x.device)
    held.index_reduce_(0, page_of, off, "amin")  # slots of earlier tokens in each touched page
    touched = torch.zeros(n_pages, dtype=torch.bool, device=x.device).index_fill_(0, page_of, True)
    grown = torch.where((held > 0)[:, None], torch.maximum(scale, need), need)
    grown = torch.where(touched[:, None], grown, scale)
    which = touched.nonzero()[:, 0]
    old = pages[which].float()
    earlier = torch.arange(size, device=x.device) < held[which][:, None]
    ratio = torch.where(earlier[:, None, :], (scale[which] / grown[which])[:, :, None], 1.0)
    pages[which] = (old * ratio[..., None]).to(pages.dtype)
    scale.copy_(grown)
    pages.view(torch.uint8)[page_of, :, off] = (x / grown[page_of][:, :, None]).to(pages.dtype).view(torch.uint8)


def _append_plain(s):
    case = s["case"]
    T, page = s["q"].shape[0], case["page"]
    b, pos = _where(s, T)
    k = _rotated(s["k"], pos, s["cos"], s["sin"], case["rot"], case["interleaved"])
    q = _rotated(s["q"], pos, s["cos"], s["sin"], case["rot"], case["interleaved"]).to(torch.bfloat16)
    page_of, off = s["block_table"][b, pos // page].long(), pos % page
    if case["cache"] == "bf16":
        s["k_pages"][page_of, :, off] = k.to(torch.bfloat16)
        s["v_pages"][page_of, :, off] = s["v"]
        return q, s["k_pages"], s["v_pages"]
    _append_e4m3(s["k_pages"], s["k_scale"], k, page_of, off)
    _append_e4m3(s["v_pages"], s["v_scale"], s["v"].float(), page_of, off)
    return q, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _attend(s, dtype):
    """Attention over the padded batch in `dtype`: O [T, Hq, d] and natural-log LSE [T, Hq], not rounded."""
    case = s["case"]
    q = s["q"].to(dtype)
    T, Hq, d = q.shape
    B, Hkv, Q = case["B"], case["Hkv"], s["max_q"]
    G = Hq // Hkv
    table = s["block_table"].long()
    L = table.shape[1] * case["page"]

    def contiguous(pages, scale):
        x = pages[table].to(dtype) if scale is None else pages[table].to(dtype) * scale[table].to(dtype)[..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, d)

    k, v = contiguous(s["k_pages"], s["k_scale"]), contiguous(s["v_pages"], s["v_scale"])
    b, pos = _where(s, T)
    i = torch.arange(T, device=q.device) - s["cu_q"].long()[b]
    padded = torch.zeros(B, Q, Hq, d, dtype=dtype, device=q.device)
    padded[b, i] = q
    padded = padded.reshape(B, Q, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, d)
    score = padded @ k.transpose(2, 3)
    score = score.mul_(1.0 / math.sqrt(d)).reshape(B, Hkv, Q, G, L)
    n = s["seq_lens"].long()
    new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    last = (n - new)[:, None] + torch.arange(Q, device=q.device)  # the last key that row i sees
    last = torch.minimum(last, n[:, None] - 1)
    hidden = torch.arange(L, device=q.device) > last[:, :, None]
    score.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(dim=-1, keepdim=True)
    out = (score.reshape(B, Hkv, Q * G, L) @ v).reshape(B, Hkv, Q, G, d) / total
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, d)[b, i]
    lse = lse.permute(0, 2, 1, 3).reshape(B, Q, Hq)[b, i]
    return out, lse


def run(state):
    s = state
    if own:
        from exact_attention_159_b200 import api
        if s["case"]["op"] == "attend":
            return api.fa_fwd_paged(s["q"], s["cache"], s["batch"], causal=True)
        q = api.fa_cache_append(s["k"], s["v"], s["cache"], s["batch"], cos=s["cos"], sin=s["sin"],
                                interleaved=s["case"]["interleaved"], q=s["q"])
        held = (s["k_pages"], s["v_pages"])
        return (q,) + (held if s["k_scale"] is None else held + (s["k_scale"], s["v_scale"]))
    if s["case"]["op"] == "append":
        return _append_plain(s)
    out, lse = _attend(s, torch.float32)
    return out.to(torch.bfloat16), lse


def work(case):
    q, n = (x.astype(np.float64) for x in _lengths(case))
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    held = 2 if case["cache"] == "bf16" else 1
    T = float(q.sum())
    touched = float((np.ceil(n / page) - np.floor((n - q) / page)).sum())
    if case["op"] == "append":
        scales = 0 if held == 2 else 2 * 2 * 4 * Hkv * touched
        moved = T * 2 * Hkv * d * (2 + held) + 2 * T * Hq * d * 2 + min(T, float(n.max())) * case["rot"] * 4
        return {"bytes": moved + scales + 4 * touched + 8 * case["B"], "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    pages = float(np.ceil(n / page).sum())
    scales = 0 if held == 2 else 2 * 4 * Hkv * pages
    cache = 2 * float(n.sum()) * Hkv * d * held
    return {"bytes": cache + 2 * T * Hq * d * 2 + 4 * T * Hq + scales + 4 * pages + 8 * case["B"],
            "flops": 4 * Hq * d * float((q * (n - (q - 1) / 2)).sum())}


def _e4m3_values(x):
    """fp64 values [0, 448] and signs rounded to the nearest e4m3 value, ties to even."""
    a = np.abs(x)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -60)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, E4M3_MAX), x)


def _exact_append(case, s):
    """One sequence and page at a time, on the host, in fp64."""
    page, rot = case["page"], case["rot"]
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    k, v, q = f64(s["k"]), f64(s["v"]), f64(s["q"])
    cos, sin = f64(s["cos"]), f64(s["sin"])
    cu, seq, table = (s[x].cpu().numpy() for x in ("cu_q", "seq_lens", "block_table"))
    kp, vp = f64(s["k_pages"]), f64(s["v_pages"])
    ks, vs = (f64(s["k_scale"]), f64(s["v_scale"])) if s["k_scale"] is not None else (None, None)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))

    def turn(x, p):
        y = x.copy()
        c, n = cos[p][:, None, :], sin[p][:, None, :]
        y[..., first] = x[..., first] * c - x[..., second] * n
        y[..., second] = x[..., second] * c + x[..., first] * n
        return y

    q_out = np.empty_like(q)
    for b in range(case["B"]):
        rows = np.arange(cu[b], cu[b + 1])
        start = int(seq[b]) - len(rows)
        p = start + np.arange(len(rows))
        q_out[rows] = turn(q[rows], p)
        for pages, scale, x in ((kp, ks, turn(k[rows], p)), (vp, vs, v[rows])):
            for j in range(start // page, (int(seq[b]) - 1) // page + 1):
                mine = np.nonzero(p // page == j)[0]
                at, off = int(table[b, j]), p[mine] % page
                new = x[mine].transpose(1, 0, 2)
                if scale is None:
                    pages[at][:, off] = new
                    continue
                old = max(0, start - j * page)
                for h in range(case["Hkv"]):
                    top = np.abs(new[h]).max()
                    need = 2.0 ** max(math.ceil(math.log2(top / E4M3_MAX)), SCALE_MIN_EXP) if top > 0 else 2.0 ** SCALE_MIN_EXP
                    now = max(need, scale[at, h]) if old else need
                    if old:
                        pages[at, h, :old] = _e4m3_values(pages[at, h, :old] * (scale[at, h] / now))
                    scale[at, h] = now
                    pages[at, h, off] = _e4m3_values(new[h] / now)
    out = (q_out, kp, vp) if ks is None else (q_out, kp, vp, ks, vs)
    return tuple(torch.from_numpy(x) for x in out)


def _exact_attend(case, s):
    """One sequence and key/value head at a time, fp64, straight from the definition."""
    cu, seq = (s[x].cpu().tolist() for x in ("cu_q", "seq_lens"))
    T, Hq, d = s["q"].shape
    G, page = Hq // case["Hkv"], case["page"]
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, new = seq[b], cu[b + 1] - cu[b]
        ids = s["block_table"][b, : -(-n // page)].long()
        seen = torch.arange(n, device="cuda")[None, :] <= (n - new + torch.arange(new, device="cuda"))[:, None]
        for h in range(case["Hkv"]):
            k, v = (s[x][ids, h].double() for x in ("k_pages", "v_pages"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][ids, h].double()[:, None, None], v * s["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("tgd,nd->tgn", s["q"][cu[b]:cu[b + 1], heads].double(), k) / math.sqrt(d)
            x = torch.where(seen[:, None, :], x, -math.inf)
            z = torch.logsumexp(x, dim=-1)
            out[cu[b]:cu[b + 1], heads] = torch.einsum("tgn,nd->tgd", torch.exp(x - z[..., None]), v)
            lse[cu[b]:cu[b + 1], heads] = z
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)
