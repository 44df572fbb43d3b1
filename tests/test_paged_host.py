"""The paged cache's refusals on the host (CPU only): nothing here reaches a kernel."""
import ctypes

import pytest
import torch

from exact_attention_159_b200 import _lib, api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


A = [0x1000000 * (i + 1) for i in range(16)]  # fake, 16-byte aligned: never dereferenced by the checks


def cache(e4m3=True, **kw):
    c = dict(K=A[0], V=A[1], K_scale=A[2], V_scale=A[3], type=int(e4m3), num_pages=10, heads=2, page_size=16, d=64)
    c.update(kw)
    return _lib.CacheStruct(*(c[n] for n, _ in _lib.CacheStruct._fields_))


def batch(**kw):
    b = dict(block_table=A[4], cu_q=A[5], seq_lens=A[6], B=3, max_pages=4, max_q=5)
    b.update(kw)
    return _lib.BatchStruct(*(b[n] for n, _ in _lib.BatchStruct._fields_))


def append(lib, c=None, b=None, T=6, K=A[7], ldk=128, V=A[8], ldv=128, Q=None, ldq=0, Qo=None, ldqo=0, Hq=0, cos=None,
           sin=None, rot=0, inter=0, n_pos=0):
    c, b = c or cache(), b or batch()
    return lib.fa_cache_append(ctypes.byref(c), ctypes.byref(b), T, K, ldk, V, ldv, Q, ldq, Qo, ldqo, Hq, cos, sin, rot,
                               inter, n_pos, None)


Q_ARGS = dict(Q=A[9], ldq=256, Qo=A[10], ldqo=256, Hq=4, cos=A[11], sin=A[12], rot=64, n_pos=100)
INVALID, UNSUPPORTED, ALIGN, OK = (_lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED, _lib.FA_ERR_ALIGNMENT, _lib.FA_OK)


@pytest.mark.parametrize("bad,code", [
    (dict(c=cache(type=2)), INVALID), (dict(c=cache(d=96)), UNSUPPORTED), (dict(c=cache(d=256)), UNSUPPORTED),
    (dict(c=cache(page_size=8)), UNSUPPORTED), (dict(c=cache(page_size=48)), UNSUPPORTED),
    (dict(c=cache(num_pages=-1)), INVALID), (dict(c=cache(num_pages=0)), INVALID), (dict(c=cache(heads=-2)), INVALID),
    (dict(c=cache(num_pages=1 << 30)), UNSUPPORTED), (dict(c=cache(K=None)), INVALID),
    (dict(c=cache(K_scale=None)), INVALID), (dict(c=cache(V=A[1] + 8)), ALIGN), (dict(c=cache(V=A[0] + 64)), INVALID),
    (dict(b=batch(B=-1)), INVALID), (dict(b=batch(max_q=-1)), INVALID), (dict(b=batch(max_pages=0)), INVALID),
    (dict(b=batch(max_pages=1 << 28)), UNSUPPORTED), (dict(b=batch(cu_q=None)), INVALID), (dict(T=-1), INVALID),
    (dict(b=batch(block_table=None)), INVALID), (dict(b=batch(seq_lens=None)), INVALID),
    (dict(K=None), INVALID), (dict(ldk=120), INVALID), (dict(ldv=64), INVALID), (dict(ldk=132), ALIGN),
    (dict(K=A[7] + 8), ALIGN), (dict(V=A[0]), INVALID), (dict(K=A[4]), INVALID), (dict(Hq=4), INVALID),
    (dict(rot=8), UNSUPPORTED), (dict(rot=80), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(inter=2), INVALID),
    (dict(rot=64, cos=None, sin=A[12]), INVALID), (dict(rot=64, cos=A[11] + 4, sin=A[12], n_pos=9), ALIGN),
    (dict(n_pos=-1), INVALID), (dict(ldk=1 << 50), UNSUPPORTED),
    (dict(Q_ARGS, Qo=None), INVALID), (dict(Q_ARGS, Hq=3), INVALID), (dict(Q_ARGS, rot=0), INVALID),
    (dict(Q_ARGS, ldq=128), INVALID), (dict(Q_ARGS, ldqo=260), ALIGN), (dict(Q_ARGS, Qo=A[9] + 16), INVALID),
    (dict(Q_ARGS, Qo=A[9], ldqo=512), INVALID), (dict(Q_ARGS, Qo=A[7]), INVALID), (dict(Q_ARGS, Qo=A[0]), INVALID),
    (dict(Q_ARGS, Qo=A[2]), INVALID), (dict(Q_ARGS, Qo=A[11]), INVALID), (dict(Q_ARGS, cos=A[1]), INVALID),
])
def test_append_refusals(lib, bad, code):
    assert append(lib, **bad) == code


def test_empty_appends(lib):
    assert append(lib, T=0) == OK and append(lib, b=batch(B=0)) == OK
    assert append(lib, c=cache(heads=0)) == OK and append(lib, b=batch(max_q=0)) == OK
    assert append(lib, c=cache(d=80), T=0) == UNSUPPORTED  # what is wrong is wrong with nothing to do too
    assert lib.fa_cache_append(None, None, 1, None, 0, None, 0, None, 0, None, 0, 0, None, None, 0, 0, 0, None) == INVALID


def fwd(lib, c=None, b=None, T=6, Q=A[7], ldq=256, O=A[8], L=A[9], W=A[10], wsb=1 << 30, Hq=4, scale=0.125, causal=1):
    c, b = c or cache(), b or batch()
    return lib.fa_fwd_paged(Q, ldq, ctypes.byref(c), ctypes.byref(b), T, O, L, W, wsb, Hq, scale, causal, None)


@pytest.mark.parametrize("bad,code", [
    (dict(Hq=5), INVALID), (dict(Hq=-4), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(causal=2), INVALID), (dict(Q=None), INVALID), (dict(L=None), INVALID),
    (dict(W=None), INVALID), (dict(ldq=128), INVALID), (dict(ldq=260), ALIGN), (dict(Q=A[7] + 8), ALIGN),
    (dict(O=A[8] + 4), ALIGN), (dict(L=A[9] + 4), ALIGN), (dict(W=A[10] + 8), ALIGN), (dict(O=A[0]), INVALID),
    (dict(O=A[7]), INVALID), (dict(L=A[8]), INVALID), (dict(W=A[3]), INVALID), (dict(W=A[4]), INVALID),
    (dict(c=cache(type=-1)), INVALID), (dict(c=cache(page_size=256)), UNSUPPORTED), (dict(wsb=16), INVALID),
    (dict(c=cache(V_scale=None)), INVALID), (dict(T=1 << 30, Hq=4), UNSUPPORTED),
])
def test_attention_refusals(lib, bad, code):
    assert fwd(lib, **bad) == code


def test_empty_attention(lib):
    assert fwd(lib, T=0) == OK and fwd(lib, b=batch(B=0)) == OK and fwd(lib, b=batch(max_q=0)) == OK
    assert fwd(lib, c=cache(heads=0), Hq=0) == OK and fwd(lib, c=cache(heads=0), Hq=4) == INVALID
    c, b = cache(d=96), batch()
    assert lib.fa_fwd_paged_workspace_size(ctypes.byref(c), ctypes.byref(b), 6, 4) == 0


def test_strerror_of_the_index_status(lib):
    assert lib.fa_strerror(_lib.FA_ERR_INDEX) != b"unknown status"


# --------------------------------------------------------------------------------- the torch binding
def test_cpu_tensors_and_wrong_kinds_are_refused():
    pages = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.PagedCache(pages, pages.clone())
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        api.PagedCache(pages.float(), pages.float())
    with pytest.raises(ValueError, match="page_size"):
        api.PagedCache(pages[:, :, :8], pages[:, :, :8])
    with pytest.raises(ValueError):
        api.PagedCache(pages[0], pages[0])
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        api.PagedBatch(i(2, 3), i(3), i(2), 1)
    with pytest.raises(ValueError):
        api.PagedBatch(i(2), i(3), i(2), 1)


# ------------------------------------------------------------------ the device's plans, run on the host
def test_plans_on_the_host(tmp_path):
    """Compiles the kernels' index arithmetic (csrc/fa_paged*.cuh) for the host and runs it over many batches:
    bad lengths, rows and pages are refused, every tile of every item is in exactly one share, and every item
    that a cut divides is joined once, from exactly the slots its parts were left in."""
    import os
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "plan")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.CSRC, "-o", exe,
                    os.path.join(here, "paged_plan_host.cu")], check=True, capture_output=True, text=True)
    done = subprocess.run([exe], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout + done.stderr
    assert "ok" in done.stdout


# ------------------------------------------------ rows turned in place, and what 32 bits of a row cannot hold
QKV = 4 * 64 + 2 * 2 * 64  # a fused projection's row: 4 query heads, 2 of keys, 2 of values, d = 64


def in_place(q=0, k=256, v=384, ldk=QKV, ldv=QKV):
    return dict(Q_ARGS, Q=A[9] + 2 * q, Qo=A[9] + 2 * q, ldq=QKV, ldqo=QKV, K=A[9] + 2 * k, ldk=ldk, V=A[9] + 2 * v,
                ldv=ldv)


@pytest.mark.parametrize("bad", [
    in_place(k=0), in_place(k=248), in_place(v=128), in_place(q=128, k=64, v=384), in_place(k=QKV - 64),
    in_place(k=256 + QKV * 3, v=QKV * 2 + 200), in_place(ldk=2 * QKV), in_place(ldv=1024),
])
def test_keys_and_values_among_queries_turned_in_place_are_refused(lib, bad):
    """Rows of K or V that share elements with the queries written in place (or are laid out so that they may)."""
    assert append(lib, **bad) == INVALID


@pytest.mark.parametrize("good", [in_place(), in_place(q=256, k=0, v=128), in_place(q=128, k=0, v=384)])
def test_a_fused_projection_is_turned_in_place(lib, good):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    assert append(lib, **good) == _lib.FA_ERR_CUDA  # the checks pass; there is no device here


def test_rows_too_wide_for_32_bits(lib):
    wide = 1 << 25
    assert append(lib, c=cache(heads=wide, num_pages=4), ldk=wide * 64, ldv=wide * 64) == UNSUPPORTED
    assert fwd(lib, T=2, Hq=wide, ldq=wide * 64) == UNSUPPORTED


def test_max_q_must_fit_32_bits():
    class Fake:  # the check comes before any tensor is looked at closely
        shape = (2, 3)

        def dim(self):
            return 2
    for bad in (-1, 1 << 31, (1 << 32) + 1):
        with pytest.raises(ValueError, match="max_q"):
            api.PagedBatch(Fake(), None, None, bad)


# ------------------------------------------------------------------- sequences that an append leaves out
def run_on_the_host(source, tmp_path, *flags):
    """Compiles a host program of this folder with the kernels' headers and runs it."""
    import os
    import subprocess
    exe = str(tmp_path / "program")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.CSRC, "-o", exe, os.path.join(here, source),
                    *flags], check=True, capture_output=True, text=True)
    done = subprocess.run([exe], capture_output=True, text=True)
    assert done.returncode == 0 and "ok" in done.stdout, done.stdout + done.stderr


def test_lengths_that_an_append_leaves_out(tmp_path):
    """Beyond the block table by one token or by far, below zero, below the new tokens: no row is taken."""
    run_on_the_host("paged_append_host.cu", tmp_path)


# ------------------------------------------------------------- what an append writes overlaps nothing else
passes = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
SCALES, PAGES = 10 * 2 * 4, 10 * 2 * 16 * 64  # bytes of the cache() above: a scale tensor, e4m3 pages


@pytest.mark.parametrize("bad", [
    dict(c=cache(V_scale=A[2])), dict(c=cache(V_scale=A[2] + SCALES - 4)), dict(c=cache(K_scale=A[3] + 4)),
    dict(c=cache(K_scale=A[0])), dict(c=cache(K_scale=A[0] + PAGES - 4)), dict(c=cache(K_scale=A[1] + 64)),
    dict(c=cache(V_scale=A[0] + 64)), dict(c=cache(V_scale=A[1] - SCALES + 4)),
    dict(b=batch(block_table=A[0])), dict(b=batch(block_table=A[1] + PAGES - 4)), dict(b=batch(block_table=A[2])),
    dict(b=batch(cu_q=A[0] + 16)), dict(b=batch(cu_q=A[3])), dict(b=batch(seq_lens=A[1])), dict(b=batch(seq_lens=A[2] - 8)),
    dict(c=cache(e4m3=False), b=batch(seq_lens=A[0] + PAGES)),  # bf16 pages are twice as large
])
def test_appends_whose_written_ranges_overlap_are_refused(lib, bad):
    """One scale tensor for keys and values (each would be stored over the other), scales among pages, pages or scales
    among the index arrays."""
    assert append(lib, **bad) == INVALID
    assert append(lib, **dict(Q_ARGS, **bad)) == INVALID


@passes
@pytest.mark.parametrize("good", [
    dict(c=cache(V_scale=A[2] + SCALES)), dict(c=cache(K_scale=A[0] + PAGES)), dict(b=batch(block_table=A[0] + PAGES)),
    dict(c=cache(e4m3=False, K_scale=A[2], V_scale=A[2])), dict(c=cache(e4m3=False, K_scale=A[0], V_scale=A[1])),
])
def test_appends_whose_ranges_meet_or_are_not_used_pass_the_checks(lib, good):
    assert append(lib, **good) == _lib.FA_ERR_CUDA


@passes
def test_attention_reads_one_scale_tensor_for_both(lib):
    assert fwd(lib, c=cache(V_scale=A[2])) == _lib.FA_ERR_CUDA


@passes
def test_an_append_with_queries_of_no_heads_is_not_empty(lib):
    """Q with zero heads has nothing to turn, but there are keys and values to append."""
    assert append(lib, **dict(Q_ARGS, Hq=0)) == _lib.FA_ERR_CUDA  # the checks pass; there is no device here
    assert append(lib, **dict(Q_ARGS, Hq=0, ldq=0, ldqo=0)) == _lib.FA_ERR_CUDA


def test_queries_of_no_heads_are_checked_like_others(lib):
    assert append(lib, **dict(Q_ARGS, Hq=0, Qo=None)) == INVALID
    assert append(lib, **dict(Q_ARGS, Hq=0, K=A[0])) == INVALID
    assert append(lib, **dict(Q_ARGS, Hq=0), T=0) == OK
    assert fwd(lib, Hq=0) == OK


# ------------------------------------------------------------------------------------- the workspace
def test_workspace_sizes_follow_the_cache_type(lib):
    """The kernel of many rows takes more than 16 rows of a bf16 cache and more than 32 of an e4m3 one, and only a call
    that may have as many needs its parts; fa.h names what the size depends on, the type among it."""
    def size(e4m3, rows, **kw):  # rows: new tokens x query heads of a key/value head
        c, b = cache(e4m3, d=128, **kw), batch(max_q=rows)
        return lib.fa_fwd_paged_workspace_size(ctypes.byref(c), ctypes.byref(b), 40, 2)

    few, parts = size(False, 16), 2 * 148 * 256 * (128 * 4 + 8)
    for e4m3, last_few in ((False, 16), (True, 32)):
        for rows in (1, 16, 17, 32, 33, 40):
            assert size(e4m3, rows) == few + (parts if rows > last_few else 0), (e4m3, rows)
            assert size(e4m3, rows, num_pages=77) == size(e4m3, rows)
            need = size(e4m3, rows)
            args = dict(c=cache(e4m3, d=128), b=batch(max_q=rows), T=40, Hq=2, W=A[15])
            assert fwd(lib, wsb=need - 1, **args) == INVALID
            if not torch.cuda.is_available():
                assert fwd(lib, wsb=need, **args) == _lib.FA_ERR_CUDA  # the checks pass; there is no device here
    import os
    with open(os.path.join(build.ROOT, "include", "fa.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    says = text[text.index("The size depends on"):]
    assert "type" in says[:says.index(" only")]


# ---------------------------------------------------------------------------------- what a handle stands for
@pytest.fixture
def handles(monkeypatch):
    """A cache and a batch of host tensors, for the binding's own checks: no call gets as far as a device."""
    monkeypatch.setattr(api, "_need", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pages = [torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
    return api.PagedCache(*pages, torch.ones(4, 2), torch.ones(4, 2)), api.PagedBatch(i(2, 3), i(3), i(2), 1)


def test_handles_are_not_changed_without_effect(handles):
    """The library is told what the handle was made of: assigning to it would change nothing of the next call."""
    for handle, names in zip(handles, (("k_pages", "v_pages", "k_scale", "v_scale", "num_pages", "page_size"),
                                       ("block_table", "cu_q", "seq_lens", "max_q", "B", "max_pages"))):
        for name in names:
            was = getattr(handle, name)
            with pytest.raises(AttributeError, match=name):
                setattr(handle, name, was + 1 if isinstance(was, int) else was.clone())
            assert getattr(handle, name) is was
    batch = handles[1]
    batch.seq_lens += 1  # in place, and the same tensor assigned again
    batch.max_q = batch.max_q
    assert batch.seq_lens.tolist() == [1, 1]


@pytest.mark.parametrize("which,name", [(0, "k_pages"), (0, "v_pages"), (0, "k_scale"), (0, "v_scale"), (1, "block_table"),
                                        (1, "cu_q"), (1, "seq_lens")])
def test_tensors_that_have_left_their_memory_are_refused(handles, which, name):
    t = getattr(handles[which], name)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    t.data = torch.zeros_like(t)  # as a tensor resized in place: the memory that was described may be another's by now
    with pytest.raises(ValueError, match="memory"):
        api.fa_cache_append(x, x, *handles)
    with pytest.raises(ValueError, match="memory"):
        api.fa_fwd_paged(x, *handles)


# ------------------------------------------------------------------------------- tensor maps kept by the host
def test_many_caches_do_not_put_out_the_other_calls_tensor_maps(lib):
    """A model has a cache for each layer and every cache its maps: the maps that the contiguous forward and backward
    reuse from call to call stay beside any number of them."""
    class Key(ctypes.Structure):  # fa_host::MapKey
        _fields_ = [("base", ctypes.c_void_p)] + [(n, ctypes.c_int) for n in ("BH", "N", "d", "rows", "kind")]

    store = getattr(lib, "_ZN7fa_host9map_storeERKNS_6MapKeyERK14CUtensorMap_st")
    lookup = getattr(lib, "_ZN7fa_host10map_lookupERKNS_6MapKeyEP14CUtensorMap_st")
    store.argtypes = lookup.argtypes = [ctypes.POINTER(Key), ctypes.c_void_p]
    store.restype, lookup.restype = None, ctypes.c_bool
    room = (ctypes.c_uint8 * 512)()
    at = -(-ctypes.addressof(room) // 64) * 64  # a tensor map is 128 bytes, aligned to 64
    base = 0x7000_0000_0000
    operand = lambda i: Key(base + i, 16, 1024, 128, 128, i % 2)  # noqa: E731  kinds 0 and 1: q, k, v, dO; dQ's sums
    pages = lambda i: Key(base + (1 << 20) + i, 80, 64, 128, 64, 2 + i % 2)  # noqa: E731  kinds 2 and 3

    def put(key, byte):
        ctypes.memset(at, byte, 128)
        store(key, at)

    def has(key, byte):
        ctypes.memset(at + 128, 0, 128)
        return lookup(key, at + 128) and ctypes.string_at(at + 128, 128) == bytes([byte]) * 128

    for i in range(20):
        put(operand(i), i + 1)
    for i in range(160):  # 80 caches, K and V
        put(pages(i), 200 - i)
    assert all(has(operand(i), i + 1) for i in range(20))
    assert has(pages(159), 200 - 159) and not has(pages(0), 200)
    for i in range(20, 200):
        put(operand(i), i + 1)
    assert has(pages(159), 200 - 159)
