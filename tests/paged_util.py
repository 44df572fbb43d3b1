"""Shared by the tests of the paged key/value cache: batches with pages handed out in no order, and a plain
64-bit implementation of both operators, one sequence at a time on the CPU, that shares no code with them.

Attention tolerances, per output element (all from the arithmetic, none from a run).  With u = 2^-8 for a
bf16 cache and 2^-11 for an e4m3 one (half a step of the type the weights P are rounded to; below 2^-14 a
half's step is absolute, at most 2^-25 of the largest weight) and A = sum_j softmax_j |v_j|:
  weights' rounding          u * A  (+ 2^-25 * sum_j |v_j| / l for halves, l >= 1 in units of the largest weight)
  the output's rounding      2^-8 * |O|
  scores: d products summed in fp32 (each addition off by at most 2^-23 of the sum of magnitudes s1), the
    products with the factors, the exponent's argument and the approximate 2^x (2^-22): ds below, which moves
    numerator and denominator alike, 2 * ds * A.  For an e4m3 cache a query row is held as a power of two times
    halves (off by 2^-25 of the row's largest magnitude) or two e4m3 parts (the second's least step is 2^-9 in units
    where the largest is 128 to 256: off by half of that, at most 2^-17 of the largest): another
    2^-17 max|q| sum|k| scale in ds
  sums and joins: fp32 relative 2^-23 per addition of a partial result, at most n_add of them
LSE: ds + 2^-22 * (n_add + |LSE|).
"""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


class Batch:
    """Host description of a ragged batch with its pages; `dev()` gives the product's handles."""

    def __init__(self, q_lens, lens, Hq, Hkv, d, page, e4m3, seed, *, extra_rows=0, extra_pages=3, kscale=None,
                 vscale=None, dead=float("nan"), share_first=False, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.lens = list(q_lens), list(lens)
        self.B, self.Hq, self.Hkv, self.G, self.d, self.page, self.e4m3 = len(lens), Hq, Hkv, Hq // Hkv, d, page, e4m3
        used = [-(-max(n, 0) // page) for n in lens]
        self.n_pages = sum(used) + extra_pages
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.max_pages = max_pages or max(1, max(used))
        self.table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)  # entries behind the last are not read
        for b, u in enumerate(used):
            for i in range(u):
                self.table[b, i] = self.table[0, 0] if share_first and i == 0 and b > 0 else order.pop()
        self.cu_q = torch.tensor([0] + list(np.cumsum(self.q_lens)), dtype=torch.int32)
        self.T_live = int(self.cu_q[-1])
        self.T = self.T_live + extra_rows
        shape = (self.n_pages, Hkv, page, d)
        self.k, self.v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        self.ks = self.vs = None
        if e4m3:
            self.ks = torch.exp2(torch.randint(-9, -6, (self.n_pages, Hkv), generator=g).float()) if kscale is None else kscale(self, g)
            self.vs = torch.exp2(torch.randint(-10, -5, (self.n_pages, Hkv), generator=g).float()) if vscale is None else vscale(self, g)
            # codes over e4m3's whole range: normals up to about 448 and some subnormals
            self.k = (self.k * 100).clamp(-448, 448).to(E4M3)
            self.v = (self.v * torch.exp2(torch.randint(-9, 8, shape, generator=g).float())).clamp(-448, 448).to(E4M3)
        else:
            self.k, self.v = self.k.bfloat16(), self.v.bfloat16()
        if dead is not None:  # what no live token owns must not matter
            owned = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for p in range(max(n, 0)):
                    owned[self.table[b, p // page], p % page] = True
            mask = ~owned[:, None, :, None].expand(shape)
            for x in (self.k, self.v):
                bits = torch.uint8 if e4m3 else torch.int16
                x.view(bits)[mask] = torch.tensor([dead]).to(x.dtype).view(bits)
        self.q = torch.randn((self.T, Hq, d), generator=g).bfloat16()

    def dev(self, max_q=None, stride=None):
        """Device copies and handles (api.PagedCache, api.PagedBatch, q)."""
        from exact_attention_159_b200 import api
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        self.dks, self.dvs = (self.ks.cuda(), self.vs.cuda()) if self.e4m3 else (None, None)
        cache = api.PagedCache(self.dk, self.dv, self.dks, self.dvs)
        batch = api.PagedBatch(self.table.cuda(), self.cu_q.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                               max(self.q_lens) if max_q is None else max_q)
        return cache, batch, self.q.cuda()

    def contiguous(self, b, h):
        """fp64 keys and values [len, d] of sequence b, key/value head h."""
        n = max(self.lens[b], 0)
        ids = self.table[b, : -(-n // self.page)].long()
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            y = x[ids, h].double()
            if s is not None:
                y = y * s[ids, h].double()[:, None, None]
            out.append(y.reshape(-1, self.d)[:n])
        return out


def reference(bt: Batch, scale, causal):
    """O, LSE [T_live, Hq(, d)] in fp64 with the tolerances tol_o, tol_lse of every element."""
    T, Hq, d = bt.T_live, bt.Hq, bt.d
    O, L = torch.zeros(T, Hq, d, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tO, tL = torch.zeros_like(O), torch.zeros_like(L)
    u = 2.0 ** -11 if bt.e4m3 else 2.0 ** -8
    for b in range(bt.B):
        n, m = max(bt.lens[b], 0), bt.q_lens[b]
        rows = slice(int(bt.cu_q[b]), int(bt.cu_q[b]) + m)
        last = torch.full((m,), n - 1) if not causal else n - m + torch.arange(m)
        seen = torch.arange(n)[None, :] <= last[:, None]
        some = seen.any(dim=1)
        for h in range(bt.Hkv):
            k, v = bt.contiguous(b, h)
            for hq in range(h * bt.G, (h + 1) * bt.G):
                q = bt.q[rows, hq].double()
                s = torch.where(seen, q @ k.T * scale, -math.inf)
                lse = torch.logsumexp(s, dim=1) if n else torch.full((m,), -math.inf, dtype=torch.float64)
                p = torch.where(some[:, None], torch.exp(s - torch.where(some, lse, 0.0)[:, None]), 0.0)
                o = p @ v
                a = p @ v.abs()
                s1 = (q.abs() @ k.abs().T).amax(dim=1) * scale if n else torch.zeros(m, dtype=torch.float64)
                top = torch.where(seen, s.abs(), 0.0).amax(dim=1) if n else torch.zeros(m, dtype=torch.float64)
                ds = (d + 8) * 2.0 ** -23 * s1 + 2.0 ** -22 * (2 * top + 64)
                if bt.e4m3 and n:
                    ds = ds + 2.0 ** -17 * q.abs().amax(dim=1) * k.abs().sum(dim=1).max() * scale
                n_add = 16 + n / 256
                tiny = 0.0
                if bt.e4m3 and n:  # halves below 2^-14 of the row's largest w_j = p_j * value scale
                    per = bt.vs[bt.table[b, : -(-n // bt.page)].long(), h].double().repeat_interleave(bt.page)[:n]
                    w = (p * per).amax(dim=1, keepdim=True)
                    tiny = 2.0 ** -25 * w * (v.abs() / per.clamp(min=2.0 ** -100)[:, None]).sum(dim=0)
                O[rows, hq], L[rows, hq] = o, lse
                tO[rows, hq] = u * a + tiny + 2.0 ** -8 * o.abs() + 2 * ds[:, None] * a + n_add * 2.0 ** -22 * a + 1e-30
                tL[rows, hq] = torch.where(some, ds + 2.0 ** -22 * (n_add + torch.where(some, lse.abs(), 0.0)), 0.0)
    return O, L, tO, tL


def check(bt: Batch, out, lse, scale, causal, label=""):
    O, L, tO, tL = reference(bt, scale, causal)
    o, l = out[: bt.T_live].double().cpu(), lse[: bt.T_live].double().cpu()
    none = torch.isneginf(L)
    assert torch.equal(torch.isneginf(l), none), f"{label}: rows without a key"
    assert bool((o[none] == 0).all()), f"{label}: O of rows without a key"
    assert bool(torch.isfinite(o).all()), f"{label}: O not finite"
    eo = ((o - O).abs() / tO).max().item() if O.numel() else 0.0
    el = ((l - L).abs()[~none] / tL[~none]).max().item() if bool((~none).any()) else 0.0
    print(f"[{label}] O {eo:.3f} of its tolerance, LSE {el:.3f}")
    assert eo <= 1.0 and el <= 1.0, (label, eo, el)


# ------------------------------------------------------------------------------------- the append
def e4m3_round(x: np.ndarray) -> np.ndarray:
    """fp64 to the nearest e4m3 value, ties to even, saturating; NaN stays."""
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where((a > 0) & np.isfinite(a), a, 1.0)))
        step = np.exp2(np.maximum(e, -6.0) - 3.0)
        r = np.where(np.isinf(a), 448.0, np.minimum(np.rint(a / step) * step, 448.0))
    return np.copysign(np.where(np.isnan(x), np.nan, r), x)


def needed_scale(amax: float) -> float:
    if amax == 0:
        return 2.0 ** -100
    m, e = math.frexp(amax)
    return 2.0 ** max(e - 9 if m <= 0.875 else e - 8, -100)


def rotate(x: np.ndarray, pos, cos, sin, interleaved):
    """fp64 rotation of [T, H, d] rows at positions pos, and the sum of magnitudes that bounds fp32's error."""
    rot = 2 * cos.shape[1]
    y, mag = x.copy(), np.abs(x)
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    c, s = cos[pos][:, None, :], sin[pos][:, None, :]
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    mag[..., i] = np.abs(x[..., i] * c) + np.abs(x[..., j] * s)
    mag[..., j] = np.abs(x[..., j] * c) + np.abs(x[..., i] * s)
    return y, mag
