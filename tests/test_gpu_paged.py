"""GPU tests of the paged key/value cache: fa_cache_append and fa_fwd_paged against plain 64-bit
implementations (tests/paged_util.py, where the tolerances are derived), at the lengths, masks, layouts and
index arrays where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from exact_attention_159_b200 import _lib, api, build
from tests.paged_util import E4M3, Batch, check, e4m3_round, needed_scale, reference, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    yield
    torch.cuda.synchronize()
    assert api.fa_last_device_status() == (0, 0)


def attend(bt, causal=True, scale=None, **kw):
    cache, batch, q = bt.dev(**kw)
    scale = 1.0 / math.sqrt(bt.d) if scale is None else scale
    out, lse = api.fa_fwd_paged(q, cache, batch, scale, causal)
    torch.cuda.synchronize()
    assert api.fa_last_device_status() == (0, 0)
    return out, lse, scale


LENS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page,Hkv,G", [(128, 16, 2, 4), (128, 64, 1, 8), (64, 32, 3, 1), (64, 128, 2, 7),
                                          (128, 128, 1, 16), (64, 16, 1, 16), (128, 32, 2, 5)])
def test_single_tokens(e4m3, d, page, Hkv, G):
    bt = Batch([1] * len(LENS), LENS, Hkv * G, Hkv, d, page, e4m3, seed=d + page + G)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"tokens d{d} p{page} {Hkv}x{G} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width", [None, 4000])
def test_short_caches_whole_or_cut(e4m3, d, width):
    """The same batch with a table just wide enough and with a wide one: items taken whole, and cut."""
    lens = [1, 7, 64, 65, 130, 200]
    bt = Batch([1] * 6, lens, 8, 2, d, 64, e4m3, seed=5, max_pages=width)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"short d{d} width {width}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page,G", [(128, 64, 4), (64, 16, 8), (128, 16, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_few_and_many_tokens(e4m3, d, page, G, causal):
    q_lens = [1, 2, 3, 0, 5, 16, 17, 40, 64, 65, 130, 1]
    lens = [300, 2, 150, 90, 5, 100, 17, 333, 64, 200, 131, 1]
    bt = Batch(q_lens, lens, 2 * G, 2, d, page, e4m3, seed=17 + G)
    out, lse, scale = attend(bt, causal)
    check(bt, out, lse, scale, causal, f"ragged d{d} p{page} G{G} causal={causal} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_no_key(e4m3, causal):
    """Sequences of length zero, and (causal) shorter than their new tokens: O = 0, LSE = -inf."""
    bt = Batch([1, 3, 2, 1, 140, 70], [0, 0, 40, 5, 33, 1], 8, 2, 128, 16, e4m3, seed=3)
    out, lse, scale = attend(bt, causal)
    check(bt, out, lse, scale, causal, f"empty rows causal={causal} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 128)])
def test_long_axis_is_cut_and_joined(e4m3, d, page):
    bt = Batch([1, 1, 2], [40001, 70, 9000], 8, 2, d, page, e4m3, seed=8, dead=None)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"long d{d} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_chunk_over_an_earlier_cache(e4m3):
    bt = Batch([500, 1, 259], [1777, 900, 259], 8, 2, 128, 32, e4m3, seed=12)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"chunk e4m3={e4m3}")


def test_prompt_chunk_d64_many_heads():
    for e4m3 in (False, True):
        bt = Batch([300, 77], [1500, 640], 24, 3, 64, 16, e4m3, seed=13)
        out, lse, scale = attend(bt)
        check(bt, out, lse, scale, True, f"chunk d64 e4m3={e4m3}")


def test_more_sequences_than_threads():
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 90, 401).tolist()
    q_lens = np.minimum(rng.integers(0, 3, 401), lens).tolist()
    bt = Batch(q_lens, lens, 4, 1, 64, 16, True, seed=2)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, "401 sequences")


@pytest.mark.parametrize("q_lens,lens", [([1, 1], [500, 300]), ([130, 64], [500, 300])])
def test_scales_far_apart(q_lens, lens):
    """Page scales of any size, among them not powers of two, zero, and values 2^40 apart."""
    def vscale(bt, g):
        s = torch.exp2(torch.randint(-20, 21, (bt.n_pages, bt.Hkv), generator=g).float()) * 1.37
        s[bt.table[0, 1].long(), 0] = 0.0
        return s

    def kscale(bt, g):
        s = torch.rand((bt.n_pages, bt.Hkv), generator=g) * 0.02
        s[bt.table[0, 2].long(), 0] = 0.0
        return s

    bt = Batch(q_lens, lens, 8, 2, 128, 32, True, seed=21, kscale=kscale, vscale=vscale)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"scales {q_lens}")


@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** -30, 2.0 ** -118, 3.0e37])
@pytest.mark.parametrize("q_lens,lens", [([1, 3], [200, 129]), ([20, 70], [300, 129])])
def test_queries_of_any_size(factor, q_lens, lens):
    """An e4m3 cache's queries become halves, or two e4m3 parts, by a power of two per row: none overflows or
    vanishes."""
    bt = Batch(q_lens, lens, 4, 1, 128, 64, True, seed=22)
    bt.q = (bt.q.float() * factor).bfloat16()
    out, lse, scale = attend(bt, scale=1.0 / math.sqrt(128) / factor)
    check(bt, out, lse, scale, True, f"queries x {factor}")


@pytest.mark.parametrize("q_lens,lens", [([1, 3], [200, 129]), ([20, 70], [300, 129])])
def test_queries_with_outliers(q_lens, lens):
    """A few columns of the queries 2^7 larger than the others, which still count."""
    for d in (64, 128):
        bt = Batch(q_lens, lens, 4, 1, d, 32, True, seed=23)
        bt.q[..., 3::29] *= 128
        bt.k.view(torch.uint8)[..., 3::29] &= 0x87  # and these columns of the keys among e4m3's subnormals
        out, lse, scale = attend(bt)
        check(bt, out, lse, scale, True, f"outliers d{d} {q_lens}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 8), (128, 1)])
def test_row_counts_about_the_tiles(e4m3, d, G):
    """Rows (new tokens x query heads) about 16, 32, 128, 256 and 384, over one to a few key tiles."""
    counts = [16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 384, 385]
    q_lens = sorted({-(-c // G) for c in counts})
    lens = [q + extra for q, extra in zip(q_lens, [0, 1, 90, 128, 129, 300, 0, 7, 255, 256, 1000, 64, 3])]
    bt = Batch(q_lens, lens, G, 1, d, 32, e4m3, seed=24)
    for causal in (True, False):
        out, lse, scale = attend(bt, causal)
        check(bt, out, lse, scale, causal, f"row counts d{d} G{G} causal={causal} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 1, 200]])
def test_pages_shared_between_sequences(e4m3, q_lens):
    bt = Batch(q_lens, [220, 90, 333], 8, 2, 128, 64, e4m3, seed=31, share_first=True)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"shared prefix e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1], [300, 20]])
def test_rows_behind_the_batch_and_strided_queries(e4m3, q_lens):
    bt = Batch(q_lens, [310, 65], 8, 2, 64, 16, e4m3, seed=32, extra_rows=9)
    cache, batch, q = bt.dev(max_q=max(q_lens) + 5)
    wide = torch.randn(bt.T, 8 + 4, 64, device="cuda").bfloat16()
    wide[:, :8] = q
    out = torch.full((bt.T, 8, 64), 7.0, device="cuda").bfloat16()
    lse = torch.full((bt.T, 8), 7.0, device="cuda")
    api.fa_fwd_paged(wide[:, :8], cache, batch, 0.125, True, out=out, lse=lse)
    torch.cuda.synchronize()
    check(bt, out, lse, 0.125, True, "strided queries")
    assert bool((out[bt.T_live:] == 7).all()) and bool((lse[bt.T_live:] == 7).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [33, 64, 128])
def test_wide_groups(e4m3, G):
    """Multi-query attention: single tokens whose query heads alone are more rows than a decode item holds."""
    bt = Batch([1, 1, 3], [700, 45, 130], G, 1, 64, 32, e4m3, seed=33)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"G {G} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1], [200, 30]])
def test_cache_beyond_32_bit_offsets(e4m3, q_lens):
    """Pages whose bytes (and elements) lie beyond 2^32 of the pool: attention, and appends to them."""
    bt = Batch(q_lens, [260, 100], 8, 8, 128, 128, e4m3, seed=34, dead=None)
    n = 2 ** 32 // (8 * 128 * 128) + 40
    far = n - 1 - torch.arange(bt.n_pages)  # the small pool's pages at the large one's end
    big = []
    for x in (bt.k, bt.v):
        y = torch.empty((n, 8, 128, 128), dtype=x.dtype, device="cuda")
        y[far.cuda()] = x.cuda()
        big.append(y)
    scales = [None, None]
    if e4m3:
        for i, x in enumerate((bt.ks, bt.vs)):
            scales[i] = torch.zeros((n, 8), device="cuda")
            scales[i][far.cuda()] = x.cuda()
    cache = api.PagedCache(*big, *scales)
    table = torch.where(bt.table >= 0, n - 1 - bt.table, bt.table)
    batch = api.PagedBatch(table.cuda(), bt.cu_q.cuda(), torch.tensor(bt.lens, dtype=torch.int32).cuda(), max(q_lens))
    out, lse = api.fa_fwd_paged(bt.q.cuda(), cache, batch, 0.1)
    assert _status() == (0, 0)
    check(bt, out, lse, 0.1, True, f"far pages e4m3={e4m3}")
    small, sb, _ = bt.dev()
    k, v = (torch.randn(bt.T, 8, 128, device="cuda").bfloat16() for _ in range(2))
    api.fa_cache_append(k, v, cache, batch)
    api.fa_cache_append(k, v, small, sb)
    assert _status() == (0, 0)
    bits = torch.uint8 if e4m3 else torch.int16
    for y, x in zip(big, (bt.dk, bt.dv)):
        assert torch.equal(y[far.cuda()].view(bits), x.view(bits))


@pytest.mark.parametrize("q_lens", [[1, 1], [200, 40]])
def test_nan_in_a_live_key_or_value_shows(q_lens):
    """It reaches rows of its own sequence as NaN, in O and LSE, and no other sequence's."""
    for which in ("k", "v"):
        for e4m3 in (False, True):
            bt = Batch(q_lens, [300, 4000], 8, 2, 128, 32, e4m3, seed=35)
            x = getattr(bt, which)
            bits = torch.uint8 if e4m3 else torch.int16
            x[int(bt.table[1, 60])].view(bits)[:, 7, 3] = torch.tensor([float("nan")]).to(x.dtype).view(bits)
            out, lse, scale = attend(bt)
            first = slice(0, q_lens[0])
            O, L, tO, tL = reference(bt, scale, True)
            assert bool(((out[first].double().cpu() - O[first]).abs() <= tO[first]).all())
            assert bool(((lse[first].double().cpu() - L[first]).abs() <= tL[first]).all())
            assert bool(out[q_lens[0]:].isnan().any())
            if which == "k":
                assert bool(lse[q_lens[0]:].isnan().all()) and bool(out[q_lens[0]:].isnan().all())


def test_empty_calls_launch_nothing():
    bt = Batch([1], [5], 4, 2, 64, 16, False, seed=1)
    cache, batch, q = bt.dev()
    out, lse = api.fa_fwd_paged(q[:0], cache, batch)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    none = api.PagedBatch(batch.block_table[:0], batch.cu_q[:1], batch.seq_lens[:0], 0)
    out = torch.full((1, 4, 64), 7.0, device="cuda").bfloat16()
    api.fa_fwd_paged(q, cache, none, out=out)
    assert bool((out == 7).all())
    k = torch.zeros((0, 2, 64), device="cuda").bfloat16()
    assert api.fa_cache_append(k, k, cache, batch) is None


# ------------------------------------------------------------------------------------ bad indices
def _status():
    torch.cuda.synchronize()
    return api.fa_last_device_status()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [200, 1, 30]])
def test_bad_indices_are_recorded_and_leave_the_other_sequences_right(e4m3, q_lens):
    lens = [260, 64, 200]
    base = Batch(q_lens, lens, 8, 2, 128, 16, e4m3, seed=41)

    def run(change):
        cache, batch, q = base.dev()
        change(batch)
        out = torch.zeros((base.T, 8, 128), device="cuda").bfloat16()
        lse = torch.zeros((base.T, 8), device="cuda")
        api.fa_fwd_paged(q, cache, batch, 0.1, True, out=out, lse=lse)
        return _status(), out, lse

    # the other sequences' results are right, not the same bits: where a sequence's keys are cut depends on
    # the lengths of all
    O, L, tO, tL = reference(base, 0.1, True)

    def right(out, lse, b):
        rows = slice(int(base.cu_q[b]), int(base.cu_q[b + 1]))
        return (bool(((out[rows].double().cpu() - O[rows]).abs() <= tO[rows]).all())
                and bool(((lse[rows].double().cpu() - L[rows]).abs() <= tL[rows]).all()))

    st, out, lse = run(lambda b: None)
    assert st == (0, 0) and all(right(out, lse, b) for b in range(3))
    for what, change in ((0xE03, lambda b: b.block_table[1].fill_(base.n_pages)),
                         (0xE03, lambda b: b.block_table[1].fill_(-1)),
                         (0xE03, lambda b: b.block_table[1].fill_(2 ** 31 - 1)),
                         (0xE02, lambda b: b.seq_lens[1].fill_(-3)),
                         (0xE02, lambda b: b.seq_lens[1].fill_(2 ** 31 - 1))):
        (rc, detail), out, lse = run(change)
        # a length far beyond the table is cut to it, where the entries behind the last token may be bad pages too
        assert rc == _lib.FA_ERR_INDEX and detail in (what, 0xE03), hex(detail)
        assert right(out, lse, 0) and right(out, lse, 2)
    (rc, detail), out, lse = run(lambda b: b.cu_q[3].fill_(base.T + 1))
    assert (rc, detail) == (_lib.FA_ERR_INDEX, 0xE01)
    assert right(out, lse, 0) and right(out, lse, 1) and bool((out[int(base.cu_q[2]):] == 0).all())
    (rc, detail), out, lse = run(lambda b: b.cu_q[0].fill_(-1))
    assert (rc, detail) == (_lib.FA_ERR_INDEX, 0xE01)
    assert _status() == (0, 0)


def test_append_bad_indices_write_nothing_of_that_token():
    bt = Batch([3, 2, 1], [40, 20, 9], 4, 2, 64, 16, True, seed=42, dead=None)
    for what, change in ((0xE03, lambda b: b.block_table[1].fill_(bt.n_pages)),
                         (0xE03, lambda b: b.block_table[1].fill_(-2)),
                         (0xE02, lambda b: b.seq_lens[1].fill_(1)),     # below its two new rows
                         (0xE02, lambda b: b.seq_lens[1].fill_(10 ** 6)),
                         (0xE01, lambda b: b.cu_q[3].fill_(99))):
        cache, batch, q = bt.dev()
        change(batch)
        k = torch.randn(6, 2, 64, device="cuda").bfloat16()
        api.fa_cache_append(k, k.clone(), cache, batch)
        rc, detail = _status()
        assert rc == _lib.FA_ERR_INDEX and detail in (what, 0xE03), hex(detail)
        for page in bt.table[1, :2].tolist():  # nothing of sequence 1's own pages moved, but where its row is still good
            if what != 0xE01:
                assert torch.equal(bt.dk[page].view(torch.uint8).cpu(), bt.k[page].view(torch.uint8))
    cache, batch, q = bt.dev()
    cos = torch.ones(38, 32, device="cuda")  # positions 38, 39 of sequence 0 are beyond the tables
    api.fa_cache_append(k, k.clone(), cache, batch, cos=cos, sin=torch.zeros_like(cos))
    assert _status() == (_lib.FA_ERR_INDEX, 0xE04)


# ---------------------------------------------------------------------------------------- append
def run_append(bt, rot, interleaved, seed, *, q_too=True, in_place=False, fused=False, spread=1.0):
    """One append and its 64-bit result; checks every byte of the pool and the rotated queries."""
    rng = np.random.default_rng(seed)
    T, Hkv, Hq, d, page = bt.T, bt.Hkv, bt.Hq, bt.d, bt.page
    new = lambda h: torch.from_numpy((rng.standard_normal((T, h, d)) * np.exp2(rng.integers(-3, 4, (T, 1, 1)) * spread))).bfloat16()  # noqa: E731
    k, v, q = new(Hkv), new(Hkv), new(Hq)
    n_pos = bt.max_pages * page
    ang = rng.uniform(0, 6.28, (n_pos, max(rot // 2, 1)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    before = [x.clone() for x in (bt.k, bt.v)] + ([bt.ks.clone(), bt.vs.clone()] if bt.e4m3 else [])
    cache, batch, _ = bt.dev()
    if fused:
        row = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], dim=1).cuda()
        qd = row[:, : Hq * d].view(T, Hq, d)
        kd, vd = (row[:, (Hq + i * Hkv) * d:(Hq + (i + 1) * Hkv) * d].unflatten(1, (Hkv, d)) for i in (0, 1))
        qd = row[:, : Hq * d].unflatten(1, (Hq, d))
    else:
        kd, vd, qd = k.cuda(), v.cuda(), q.cuda()
    kw = {}
    if rot:
        kw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(), interleaved=interleaved)
        if q_too:
            kw["q"] = qd
            if in_place:
                kw["q_out"] = qd
            else:
                kw["q_out"] = torch.full((T, Hq, d), 5.0, device="cuda").bfloat16()
    got_q = api.fa_cache_append(kd, vd, cache, batch, **kw)
    assert _status() == (0, 0)

    f64 = lambda x: x.double().numpy()  # noqa: E731
    c64, s64 = cos.astype(np.float64), sin.astype(np.float64)
    want = [f64(x).copy() for x in before[:2]]
    tol = [np.zeros_like(want[0]), np.zeros_like(want[1])]
    exact_bytes = [np.ones(want[0].shape, dtype=bool), np.ones(want[1].shape, dtype=bool)]
    scales = [f64(x).copy() for x in before[2:]]
    for b in range(bt.B):
        rows = np.arange(int(bt.cu_q[b]), int(bt.cu_q[b + 1]))
        if len(rows) == 0:
            continue
        pos = bt.lens[b] - len(rows) + np.arange(len(rows))
        for x in range(2):
            y, mag = (f64(k)[rows], None) if x == 0 else (f64(v)[rows], None)
            if x == 0 and rot:
                y, mag = rotate(y, pos, c64, s64, interleaved)
            if mag is None:
                mag = np.zeros_like(y)
            fp32 = mag * 2.0 ** -22  # two products, one addition, each half a step of fp32
            for j in sorted(set((pos // page).tolist())):
                mine = np.nonzero(pos // page == j)[0]
                at, off = int(bt.table[b, j]), pos[mine] % page
                if not bt.e4m3:
                    want[x][at][:, off] = y[mine].transpose(1, 0, 2)
                    tol[x][at][:, off] = (2.0 ** -8 * np.abs(y[mine]) * (1 if x == 0 and rot else 0) + fp32[mine]).transpose(1, 0, 2)
                    exact_bytes[x][at][:, off] = not (x == 0 and rot)
                    continue
                earlier = int(off.min())
                for h in range(Hkv):
                    fin = np.abs(y[mine, h])[np.isfinite(y[mine, h])]
                    need = needed_scale(float(fin.max()) if fin.size else 0.0)
                    now = max(need, scales[x][at, h]) if earlier else need
                    if earlier:
                        want[x][at, h, :earlier] = e4m3_round(want[x][at, h, :earlier] * (scales[x][at, h] / now))
                    scales[x][at, h] = now
                    val = y[mine, h] / now
                    want[x][at, h, off] = val
                    e = np.floor(np.log2(np.maximum(np.abs(val), 2.0 ** -30)))
                    tol[x][at, h, off] = np.exp2(np.maximum(e, -6.0) - 4.0) * (1 + 2.0 ** -20) + fp32[mine, h] / now
                    exact_bytes[x][at, h, off] = False
    for x, dev in enumerate((bt.dk, bt.dv)):
        got = dev.cpu()
        g = f64(got)
        same = exact_bytes[x]
        assert np.array_equal(g[same], want[x][same], equal_nan=True), "kv"[x] + ": slots that must be exact"
        assert (np.abs(g[~same] - want[x][~same]) <= tol[x][~same]).all(), "kv"[x] + ": new slots"
        if bt.e4m3:
            assert np.array_equal(f64((bt.dks, bt.dvs)[x].cpu()), scales[x]), "kv"[x] + ": scales"
    if rot and q_too:
        want_q = f64(q).copy()
        for b in range(bt.B):
            rows = np.arange(int(bt.cu_q[b]), int(bt.cu_q[b + 1]))
            if len(rows):
                pos = bt.lens[b] - len(rows) + np.arange(len(rows))
                want_q[rows], mag = rotate(f64(q)[rows], pos, c64, s64, interleaved)
                d_ = np.abs(f64(got_q.cpu())[rows] - want_q[rows])
                assert (d_ <= 2.0 ** -8 * np.abs(want_q[rows]) + mag * 2.0 ** -22).all()
        tail = got_q[bt.T_live:].cpu()
        assert torch.equal(tail, q[bt.T_live:] if in_place else torch.full_like(tail, 5.0)), "rows behind the batch"
    # the rest of a fused row is only read
    if fused:
        assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 32), (128, 64), (128, 128), (64, 16), (64, 32), (64, 64), (64, 128)])
@pytest.mark.parametrize("rot,interleaved", [(0, False), ("d", False), ("d", True), (16, False), (48, True)])
def test_append(e4m3, d, page, rot, interleaved):
    q_lens = [1, 1, 1, 3, 0, 17, page, page + 1, 150, 2, 40]
    lens = [1, page, page + 1, 2 * page + 2, 30, 17, page, 3 * page, 150, page + 1, 40 + page // 2]
    bt = Batch(q_lens, lens, 6, 2, d, page, e4m3, seed=7 + page + d, extra_rows=3, dead=None)
    run_append(bt, d if rot == "d" else rot, interleaved, seed=page)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_in_place_and_from_a_fused_projection(e4m3):
    for in_place, fused in ((True, False), (False, True), (True, True)):
        bt = Batch([5, 1, 70], [100, 33, 70], 8, 2, 128, 32, e4m3, seed=71, extra_rows=2, dead=None)
        run_append(bt, 128, False, seed=3, in_place=in_place, fused=fused)


def test_append_many_single_tokens_and_growing_scales():
    """Single tokens of sizes up to 2^20 apart: page scales grow, the earlier codes with them."""
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 400, 130).tolist()
    bt = Batch([1] * 130, lens, 8, 8, 128, 64, True, seed=72, dead=None)
    run_append(bt, 128, False, seed=5, spread=3.0)


def test_append_codes_of_special_values():
    """Zeros, infinities, NaN, the largest and the smallest values: scales by the finite ones alone."""
    bt = Batch([4, 4, 4, 1], [4, 4, 4, 1], 1, 1, 64, 16, True, seed=73, dead=None)
    cache, batch, _ = bt.dev()
    x = torch.zeros(13, 1, 64)
    x[0, 0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
    x[1, 0, 0] = 3.0
    x[4, 0, 0] = torch.finfo(torch.bfloat16).max
    x[8, 0, :2] = torch.tensor([2.0 ** -126, 2.0 ** -130])
    x = x.bfloat16()
    api.fa_cache_append(x.cuda(), x.cuda(), cache, batch)
    assert _status() == (0, 0)
    want = [2.0 ** -7, needed_scale(float(torch.finfo(torch.bfloat16).max)), 2.0 ** -100, 2.0 ** -100]
    for codes, scale in ((bt.dk, bt.dks), (bt.dv, bt.dvs)):
        for b, rows in enumerate((slice(0, 4), slice(4, 8), slice(8, 12), slice(12, 13))):
            page = int(bt.table[b, 0])
            assert scale[page, 0].item() == want[b]
            got = codes[page, 0, : rows.stop - rows.start].double().cpu().numpy()
            ref = e4m3_round(x[rows, 0].double().numpy() / want[b])
            assert np.array_equal(got, ref, equal_nan=True)


# ------------------------------------------------------------------------------- as they are used
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_run_of_them_prompts_then_tokens(e4m3, d):
    """Prompts in chunks, then tokens one by one: every step's attention against 64 bits over what the cache
    then holds, the cache against the keys and values given, and (bf16) the contiguous forward's result."""
    rng = torch.Generator().manual_seed(d)
    B, Hq, Hkv, page, base = 3, 8, 2, 32, 10000.0
    total = [150, 61, 203]
    steps = [[64, 30, 100], [83, 29, 100], [1, 1, 1], [1, 1, 1], [1, 0, 1]]
    done = [0] * B
    pages = sum(-(-n // page) for n in total) + 2
    order = torch.randperm(pages, generator=rng).to(torch.int32)
    width = max(-(-n // page) for n in total)
    table = torch.zeros((B, width), dtype=torch.int32)
    at = 0
    for b, n in enumerate(total):
        u = -(-n // page)
        table[b, :u] = order[at:at + u]
        at += u
    dt = E4M3 if e4m3 else torch.bfloat16
    kp, vp = (torch.full((pages, Hkv, page, d), float("nan"), device="cuda").to(dt) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), float("nan"), device="cuda") for _ in range(2)) if e4m3 else (None, None)
    cache = api.PagedCache(kp, vp, ks, vs)
    half = torch.arange(d // 2, dtype=torch.float64)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * base ** (-half / (d // 2))
    cos, sin = ang.cos().float(), ang.sin().float()
    full = [[torch.zeros(n, h, d).bfloat16() for n in total] for h in (Hq, Hkv, Hkv)]
    for new in steps:
        T = sum(new)
        q, k, v = (torch.randn(T, h, d, generator=rng).bfloat16() for h in (Hq, Hkv, Hkv))
        done = [a + b for a, b in zip(done, new)]
        cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        batch = api.PagedBatch(table.cuda(), cu.cuda(), torch.tensor(done, dtype=torch.int32).cuda(), max(new))
        qr = api.fa_cache_append(k.cuda(), v.cuda(), cache, batch, cos=cos.cuda(), sin=sin.cuda(), q=q.cuda())
        out, lse = api.fa_fwd_paged(qr, cache, batch)
        assert _status() == (0, 0)
        for b in range(B):
            rows, first = slice(int(cu[b]), int(cu[b + 1])), done[b] - new[b]
            kr, mag = rotate(k[rows].double().numpy(), first + np.arange(new[b]), cos.double().numpy(), sin.double().numpy(), False)
            full[1][b][first:done[b]] = torch.from_numpy(kr).bfloat16()
            full[2][b][first:done[b]] = v[rows]
            full[0][b][first:done[b]] = qr[rows].cpu()
        bt = Batch.__new__(Batch)
        bt.q_lens, bt.lens, bt.B, bt.Hq, bt.Hkv, bt.G, bt.d, bt.page, bt.e4m3 = new, done, B, Hq, Hkv, Hq // Hkv, d, page, e4m3
        bt.k, bt.v, bt.ks, bt.vs = kp.cpu(), vp.cpu(), None if ks is None else ks.cpu(), None if vs is None else vs.cpu()
        bt.table, bt.cu_q, bt.T_live, bt.q = table, cu, T, qr.cpu()
        check(bt, out, lse, 1.0 / math.sqrt(d), True, f"step {new} e4m3={e4m3}")
    for b in range(B):
        for h in range(Hkv):
            n = done[b]
            got_k, got_v = bt.contiguous(b, h)
            for got, want in ((got_k, full[1][b][:n, h].double()), (got_v, full[2][b][:n, h].double())):
                if e4m3:  # half a step of e4m3 by its page's scale, and once more where the scale has grown since
                    blocks = -(-n // page)
                    tol = torch.zeros(n, d, dtype=torch.float64)
                    for j in range(blocks):
                        sl = slice(j * page, min((j + 1) * page, n))
                        sc = (bt.ks if got is got_k else bt.vs)[table[b, j].long(), h].double()
                        tol[sl] = 2 * (2.0 ** -4 * want[sl].abs() + 2.0 ** -10 * sc) + 2.0 ** -8 * want[sl].abs()
                    assert bool(((got - want).abs() <= tol).all())
                else:
                    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -20).all())
    if not e4m3:
        n = done[2]
        o, l = api.fa_fwd_qk(*(full[i][2][:n].permute(1, 0, 2)[None].contiguous().cuda() for i in range(3)), causal=True)
        # the last token's row by both: each within 2 u A + u |O| of the truth, |v| < 6
        a, c = o[0, :, -1].double().cpu(), out[-1].double().cpu()
        assert float((a - c).abs().max()) <= 4 * 2.0 ** -8 * 6


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_step_replays_with_new_lengths(e4m3):
    """A decode step (append, then attention) captured once and replayed as the sequences grow."""
    bt = Batch([1, 1, 1], [40, 130, 17], 8, 2, 128, 16, e4m3, seed=51, dead=None, max_pages=12)
    for b in range(3):  # pages for the tokens to come
        for i in range(12):
            bt.table[b, i] = bt.table[b, i] if bt.table[b, i] >= 0 else 0
    spare = iter([p for p in range(bt.n_pages) if p not in set(bt.table.flatten().tolist())])
    bt.table[0, 3] = next(spare)
    bt.table[2, 2] = next(spare)
    cache, batch, q = bt.dev()
    k, v = (torch.zeros(3, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cos, sin = torch.ones(192, 64, device="cuda"), torch.zeros(192, 64, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(3, 8, device="cuda")
    qr = torch.zeros_like(q)
    ws = torch.empty(api.fa_fwd_paged_workspace_size(cache, batch, 3, 8), dtype=torch.uint8, device="cuda")

    def step():
        api.fa_cache_append(k, v, cache, batch, cos=cos, sin=sin, q=q, q_out=qr)
        api.fa_fwd_paged(qr, cache, batch, 0.1, True, out=out, lse=lse, workspace=ws)

    g = torch.Generator(device="cuda").manual_seed(9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(11):
        batch.seq_lens += 1
        bt.lens = [x + 1 for x in bt.lens]
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        ws.fill_(0xFF)
        graph.replay()
        assert _status() == (0, 0)
        bt.k, bt.v = bt.dk.cpu(), bt.dv.cpu()
        if e4m3:
            bt.ks, bt.vs = bt.dks.cpu(), bt.dvs.cpu()
        bt.q = qr.cpu()
        check(bt, out, lse, 0.1, True, f"replay {n}")


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_prompt_chunk(e4m3):
    """Prompt chunks (appends by clusters of blocks, both attention kernels and the join) in a captured graph."""
    bt = Batch([200, 1, 33], [330, 90, 33], 8, 2, 128, 128, e4m3, seed=52, dead=None)
    cache, batch, q = bt.dev()
    k, v = (torch.randn(bt.T, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cos, sin = torch.ones(512, 64, device="cuda"), torch.zeros(512, 64, device="cuda")
    out, lse, qr = torch.zeros_like(q), torch.zeros(bt.T, 8, device="cuda"), torch.zeros_like(q)
    ws = torch.empty(api.fa_fwd_paged_workspace_size(cache, batch, bt.T, 8), dtype=torch.uint8, device="cuda")

    def step():
        api.fa_cache_append(k, v, cache, batch, cos=cos, sin=sin, q=q, q_out=qr)
        api.fa_fwd_paged(qr, cache, batch, 0.1, True, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, device="cuda"))
    for n in range(3):
        ws.fill_(0xFF)
        out.zero_()
        graph.replay()
        assert _status() == (0, 0)
        bt.k, bt.v, bt.q = bt.dk.cpu(), bt.dv.cpu(), qr.cpu()
        if e4m3:
            bt.ks, bt.vs = bt.dks.cpu(), bt.dvs.cpu()
        check(bt, out, lse, 0.1, True, f"chunk replay {n} e4m3={e4m3}")


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [150, 1, 9]])
def test_same_call_gives_the_same_bits_and_streams_do_not_meet(q_lens):
    bt = Batch(q_lens, [5000, 333, 1200], 8, 2, 128, 64, True, seed=61, dead=None)
    cache, batch, q = bt.dev()
    want, wl = api.fa_fwd_paged(q, cache, batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        got.append(api.fa_fwd_paged(q, cache, batch, stream=streams[i % 2]))
        del_me = torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # noqa: F841  reuses what the current stream freed
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, wl)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_len", [1, 3, 150])
@pytest.mark.parametrize("length", [161, 170, 10 ** 6, 2 ** 31 - 1, -3, -2 ** 31])
def test_append_leaves_out_a_sequence_of_a_length_its_table_does_not_hold(e4m3, q_len, length):
    """Its table is full of valid pages, the last one shared with another sequence (as a full one may be): no byte of
    them, no scale and no query row of that sequence is written; the other sequences' tokens are."""
    bt = Batch([3, q_len, 1], [40, 160, 9], 4, 2, 64, 16, e4m3, seed=43, dead=None)
    bt.table[0, 0] = bt.table[1, 9]
    g = torch.Generator().manual_seed(q_len)
    k, v, q = (torch.randn(bt.T, h, 64, generator=g).bfloat16().cuda() * 4 for h in (2, 2, 4))
    angle = torch.rand(160, 32, generator=g).cuda()
    mine = torch.zeros(bt.T, dtype=torch.bool, device="cuda")
    mine[3:3 + q_len] = True

    def run(rows, batch, cache):
        out = torch.full((len(rows), 4, 64), 5.0, device="cuda").bfloat16()
        api.fa_cache_append(k[rows], v[rows], cache, batch, cos=angle.cos(), sin=angle.sin(), q=q[rows], q_out=out)
        return _status(), out, [x.view(torch.uint8).clone() for x in (bt.dk, bt.dv, bt.dks, bt.dvs) if x is not None]

    cache, batch, _ = bt.dev()
    batch.seq_lens[1] = length
    st, got_q, got = run(torch.arange(bt.T, device="cuda"), batch, cache)
    assert st == (_lib.FA_ERR_INDEX, 0xE02)
    assert bool((got_q[mine] == 5).all())
    cache, batch, _ = bt.dev()  # the same without that sequence's tokens
    batch.cu_q.copy_(torch.tensor([0, 3, 3, 4], dtype=torch.int32))
    st, want_q, want = run((~mine).nonzero()[:, 0], batch, cache)
    assert st == (0, 0) and torch.equal(got_q[~mine], want_q)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("big", [20, 27, 40, 60])
@pytest.mark.parametrize("order", ["zeros first", "zeros last", "alternating"])
@pytest.mark.parametrize("q_lens,lens,page", [([1, 1], [300, 257], 128), ([1, 3], [130, 250], 32), ([1, 2], [20000, 90], 64),
                                              ([70, 300], [500, 777], 32), ([20], [9000], 128), ([70], [6000], 16)])
def test_pages_of_zeros_beside_large_scales(big, order, q_lens, lens, page):
    """A page of zeros has no weight in O but all of its weight in the softmax's sum, whatever the other pages' value
    scales: over one key tile (by different warps), several, and several shares joined, in any order."""
    def vscale(bt, g):
        s = torch.full((bt.n_pages, bt.Hkv), 2.0 ** big)
        for b, n in enumerate(bt.lens):
            used = -(-n // bt.page)
            for i in range(used):
                zero = {"zeros first": i < used // 2, "zeros last": i >= (used + 1) // 2, "alternating": i % 2 == 0}[order]
                if zero:
                    s[int(bt.table[b, i])] = 0.0
        return s

    bt = Batch(q_lens, lens, 8, 2, 128, page, True, seed=25, vscale=vscale, dead=None)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"zeros beside 2^{big}, {order}, {q_lens} {lens}")


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_with_no_query_heads_appends_the_keys_and_values(e4m3):
    """Q with zero heads (given to the library by pointer) has nothing to turn; the keys and values are appended."""
    import ctypes
    bt = Batch([3, 1], [40, 17], 4, 2, 64, 16, e4m3, seed=44, dead=None)
    k, v, q = (torch.randn(4, 2, 64, device="cuda").bfloat16() for _ in range(3))
    cos, sin = torch.ones(48, 32, device="cuda"), torch.zeros(48, 32, device="cuda")
    cache, batch, _ = bt.dev()
    assert api.fa_cache_append(k, v, cache, batch, cos=cos, sin=sin) is None
    want = [bt.dk.view(torch.uint8), bt.dv.view(torch.uint8)]
    assert _status() == (0, 0)
    assert not torch.equal(want[0].cpu(), bt.k.view(torch.uint8)) and not torch.equal(want[1].cpu(), bt.v.view(torch.uint8))
    cache, batch, _ = bt.dev()
    q_out = torch.full_like(q, 5.0)
    rc = _lib.lib().fa_cache_append(cache._ref, batch._ref, 4, k.data_ptr(), 128, v.data_ptr(), 128, q.data_ptr(), 128,
                                    q_out.data_ptr(), 128, 0, cos.data_ptr(), sin.data_ptr(), 64, 0, 48,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == _lib.FA_OK and _status() == (0, 0)
    assert torch.equal(bt.dk.view(torch.uint8), want[0]) and torch.equal(bt.dv.view(torch.uint8), want[1])
    assert bool((q_out == 5).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_lens,lens,Hkv,G", [([16], [70001], 1, 8), ([64, 1], [16400, 300], 2, 4)])
def test_short_chunk_over_a_long_cache_is_joined_from_many_parts(e4m3, q_lens, lens, Hkv, G):
    """Items of the kernel of many rows cut into more parts than a warp has lanes."""
    bt = Batch(q_lens, lens, Hkv * G, Hkv, 128, 64, e4m3, seed=26, dead=None)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"many parts {q_lens} over {lens} e4m3={e4m3}")


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_single_tokens_beside_a_long_chunk(e4m3):
    """Both kernels of one call with work for every SM."""
    rng = np.random.default_rng(6)
    lens = rng.integers(100, 3000, 40).tolist()
    bt = Batch([1] * 20 + [700] + [1] * 19, lens[:20] + [2500] + lens[21:], 8, 2, 128, 32, e4m3, seed=27, dead=None)
    out, lse, scale = attend(bt)
    check(bt, out, lse, scale, True, f"tokens beside a chunk e4m3={e4m3}")


def test_many_caches_and_two_host_threads():
    """A cache for each of 40 layers (more tensor maps than the host keeps), in turn and from two threads on two
    streams: every call's bits are those of the call alone."""
    import threading
    bts = [Batch([1, 40, 1], [500, 700 + i, 33], 8, 2, 128, 32, bool(i % 2), seed=100 + i, dead=None) for i in range(40)]
    handles = [bt.dev() for bt in bts]
    want = [tuple(x.clone() for x in api.fa_fwd_paged(q, c, b, 0.1)) for c, b, q in handles]
    assert _status() == (0, 0)
    for i in (0, 1, 39):
        check(bts[i], *want[i], 0.1, True, f"cache {i}")
    same = [False, False]

    def calls(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [api.fa_fwd_paged(q, c, b, 0.1) for c, b, q in handles[k::2] * 3]
            stream.synchronize()
            same[k] = all(torch.equal(x, y) for o, w in zip(got, want[k::2] * 3) for x, y in zip(o, w))

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same) and _status() == (0, 0)


def test_handles_whose_tensors_were_resized_are_refused():
    bt = Batch([1], [40], 4, 2, 64, 16, True, seed=45)
    for which, name in ((0, "k_pages"), (0, "v_scale"), (1, "cu_q"), (1, "block_table")):
        cache, batch, q = bt.dev()
        getattr((cache, batch)[which], name).resize_(1 << 22)
        with pytest.raises(ValueError, match="memory"):
            api.fa_fwd_paged(q, cache, batch)
        with pytest.raises(ValueError, match="memory"):
            api.fa_cache_append(q[:, :2], q[:, 2:], cache, batch)
