"""The paged cache, its attention and the sampled accept refuse bad arguments on the host, before anything
is enqueued, and say what is wrong; the Python binding refuses what it can see of its tensors.

Every call below is one that validation must refuse (or that has nothing to enqueue).
"""
import ctypes
import math
import os

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.test_abi_host import Bufs, ERR_ALIAS, ERR_ALIGN, ERR_ARG, ERR_RANGE, OK, _header_constant
from tests.test_ops_host import _refused, _up


class _Cache(ctypes.Structure):   # kda_cache
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "table", "lens")] +
                [(n, ctypes.c_longlong) for n in ("page_stride", "row_stride", "head_stride")] +
                [(n, ctypes.c_int) for n in ("pages", "page_rows", "seq_pages")])


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.lib_path()):
        from gated_delta_rule_rows_amd import build
        build.build()
    return kda.load()


@pytest.fixture(scope="module")
def b():
    return Bufs()


def _cache(b, **kw):
    a = dict(k=b["k"], v=b["v"], table=b["ptrs"], lens=b["s_in"], page_stride=16 * 2 * 128, row_stride=2 * 128,
             head_stride=128, pages=4, page_rows=16, seq_pages=5)
    a.update({n: v for n, v in kw.items() if n in a})
    return _Cache(*(a[n].value if isinstance(a[n], ctypes.c_void_p) else a[n] for n, _ in _Cache._fields_))


def _append(lib, b, **kw):
    a = dict(nk=b["q"], k_ld=256, nv=b["g"], v_ld=256, off=b["s_out"], R=6, B=3, Hk=2, dt=0)
    a.update(kw)
    c = None if kw.get("cache", 1) is None else ctypes.byref(_cache(b, **kw))
    return lib.kda_cache_append(a["nk"], a["k_ld"], a["nv"], a["v_ld"], c, a["off"], a["R"], a["B"], a["Hk"], a["dt"], None)


def _attn(lib, b, **kw):
    a = dict(q=b["q"], q_ld=512, off=b["s_out"], o=b["o"], R=6, B=3, H=4, Hk=2, scale=0.1, window=0, sinks=0, dt=0,
             work=b["snap"], bytes=64 << 20)
    a.update(kw)
    c = None if kw.get("cache", 1) is None else ctypes.byref(_cache(b, **kw))
    return lib.kda_attn_rows(a["q"], a["q_ld"], c, a["off"], a["o"], a["R"], a["B"], a["H"], a["Hk"], a["scale"],
                             a["window"], a["sinks"], a["dt"], a["work"], a["bytes"], None)


def _sampled(lib, b, **kw):
    a = dict(x=b["q"], ld=100, dt=0, probs=b["k"], probs_ld=100, off=b["s_in"], d=b["v"], u=b["g"], temp=b["beta"],
             out=b["o"], p=b["s_out"], R=6, B=3, V=100, work=b["snap"], bytes=64 << 20)
    a.update(kw)
    return lib.kda_accept_sampled(a["x"], a["ld"], a["dt"], a["probs"], a["probs_ld"], a["off"], a["d"], a["u"],
                                  a["temp"], a["out"], a["p"], a["R"], a["B"], a["V"], a["work"], a["bytes"], None)


@pytest.mark.parametrize("call", [_append, _attn])
def test_cache_refusals(lib, b, call):
    def no(want, *words, **kw):
        _refused(lib, call(lib, b, **kw), want, *words)

    no(ERR_ARG, "cache is NULL", cache=None)
    no(ERR_RANGE, "cache.pages=0", pages=0)
    for rows in (0, -16, 3, 48, 2 * _header_constant("KDA_PAGE_ROWS_MAX")):
        no(ERR_RANGE, "page_rows", page_rows=rows)
    no(ERR_RANGE, "seq_pages=0", seq_pages=0)
    no(ERR_RANGE, "seq_pages", seq_pages=(1 << 26) + 1)                 # over 2^30 rows
    no(ERR_RANGE, "negative", page_stride=-4096)
    no(ERR_RANGE, "too large", page_stride=(1 << 40) + 4)
    no(ERR_RANGE, "too large", page_stride=1 << 39)
    no(ERR_ALIGN, "stride", row_stride=258)
    no(ERR_ALIGN, "stride", dt=1, head_stride=132)
    no(ERR_RANGE, "overlap", row_stride=252)
    no(ERR_RANGE, "overlap", head_stride=0)
    no(ERR_RANGE, "overlap", page_stride=4092)
    for name in ("k", "v", "table", "lens"):
        no(ERR_ARG, "cache." + name, **{name: None})
        no(ERR_ALIGN, "cache." + name, **{name: _up(b["o"], 2 if name in ("table", "lens") else 8)})
    no(ERR_ARG, "in_dtype", dt=2)
    no(ERR_RANGE, "R=-1", R=-1)
    no(ERR_RANGE, "R=", R=_header_constant("KDA_PROMPT_ROWS_MAX") + 1)
    no(ERR_RANGE, "B=0", B=0)
    no(ERR_RANGE, "B=", B=_header_constant("KDA_PROMPT_SEQS_MAX") + 1)
    no(ERR_RANGE, "H", **({"H": 0, "Hk": 1} if call is _attn else {"Hk": 0}))
    no(ERR_ARG, "offsets", off=None)
    no(ERR_ALIGN, "offsets", off=_up(b["s_out"], 2))


def test_append_refusals(lib, b):
    def no(want, *words, **kw):
        _refused(lib, _append(lib, b, **kw), want, *words)

    no(ERR_RANGE, "R=", R=1 << 24)
    no(ERR_RANGE, "k_ld=255", k_ld=255)
    no(ERR_RANGE, "v_ld=", v_ld=1 << 40)
    no(ERR_ALIGN, "k_ld=257", k_ld=257)
    no(ERR_ALIGN, "v_ld=260", v_ld=260, dt=1)
    no(ERR_ARG, "k is NULL", nk=None)
    no(ERR_ALIGN, "v is not", nv=_up(b["g"], 4))
    no(ERR_ALIAS, "cache.k overlaps k", nk=_up(b["k"], 32))
    no(ERR_ALIAS, "cache.v overlaps v", nv=b["v"])
    no(ERR_ALIAS, "cache.k overlaps offsets", off=b["k"])
    no(ERR_ALIAS, "cache.v overlaps cache.table", table=b["v"])
    no(ERR_ALIAS, "cache.k overlaps cache.lens", lens=b["k"])
    # keys and values in one buffer
    no(ERR_ALIAS, "cache.k and cache.v", v=b["k"])
    no(ERR_ALIAS, "cache.k and cache.v", v=_up(b["k"], 128 * 4))
    no(ERR_ALIAS, "cache.k and cache.v", v=_up(b["k"], 4096 * 4), page_stride=4096 + 256)
    assert _append(lib, b, R=0, nk=None, nv=None) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, v=_up(b["k"], 4096 * 4), page_stride=8192) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, v=_up(b["k"], 256 * 4), row_stride=512, page_stride=8192) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, v=_up(b["k"], 128 * 4), head_stride=256, row_stride=512, page_stride=8192) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, head_stride=16 * 128, row_stride=128) == OK
    # one page, row or head has no stride
    assert _append(lib, b, R=0, nk=None, nv=None, pages=1, page_stride=-7) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, Hk=1, head_stride=3, k_ld=128, v_ld=128) == OK
    assert _append(lib, b, R=0, nk=None, nv=None, page_rows=1, row_stride=-1, page_stride=256) == OK


def test_attn_refusals(lib, b):
    def no(want, *words, **kw):
        _refused(lib, _attn(lib, b, **kw), want, *words)

    no(ERR_RANGE, "divide H=4", Hk=3)
    no(ERR_RANGE, "H=65536", H=65536)
    for scale in (0.0, -1.0, math.nan, math.inf):
        no(ERR_RANGE, "scale", scale=scale)
    no(ERR_RANGE, "window=-1", window=-1)
    no(ERR_RANGE, "sinks=-1", sinks=-1, window=5)
    no(ERR_RANGE, "sinks=4", sinks=4)
    no(ERR_RANGE, "too many", R=1 << 28, H=64, Hk=32, q_ld=8192)
    no(ERR_RANGE, "q_ld=508", q_ld=508)
    no(ERR_ALIGN, "q_ld=514", q_ld=514)
    no(ERR_ARG, "q is NULL", q=None)
    no(ERR_ARG, "o is NULL", o=None)
    no(ERR_ALIGN, "o is not", o=_up(b["o"], 8))
    no(ERR_ALIAS, "o overlaps q", o=b["q"])
    no(ERR_ALIAS, "o overlaps cache.v", o=b["v"])
    no(ERR_ALIAS, "o overlaps cache.lens", o=b["s_in"])
    need = lib.kda_attn_rows_work_bytes(6, 3, 4, 2)
    assert need > 0
    no(ERR_RANGE, "work_bytes", str(need), bytes=need - 1)
    no(ERR_ARG, "work is NULL", work=None)
    no(ERR_ALIGN, "work", work=_up(b["snap"], 8))
    no(ERR_ALIAS, "work overlaps cache.k", work=b["k"])
    no(ERR_ALIAS, "o overlaps work", work=b["o"])
    assert _attn(lib, b, R=0, q=None, o=None) == OK


def test_attn_workspace_never_shrinks(lib):
    for H, Hk in ((1, 1), (8, 1), (64, 8), (12, 4), (130, 1), (64, 64)):
        last = 0
        for R, B in ((0, 1), (1, 1), (2, 1), (15, 1), (33, 1), (33, 20), (100, 20), (4096, 20), (4096, 900), (100000, 4096)):
            n = lib.kda_attn_rows_work_bytes(R, B, H, Hk)
            assert n >= last > -1
            last = n
        assert last < 256 << 20
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 4, 3), (1, 1, 70000, 1), (1, 5000, 1, 1)):
        assert lib.kda_attn_rows_work_bytes(*bad) == -1


def test_sampled_refusals(lib, b):
    def no(want, *words, **kw):
        _refused(lib, _sampled(lib, b, **kw), want, *words)

    no(ERR_ARG, "in_dtype", dt=7)
    no(ERR_RANGE, "R=-1", R=-1)
    no(ERR_RANGE, "B=0", B=0)
    no(ERR_RANGE, "V=0", V=0)
    no(ERR_RANGE, "V=", V=(1 << 30) + 1, ld=1 << 31)
    no(ERR_RANGE, "ld=99", ld=99)
    no(ERR_RANGE, "probs_ld=99", probs_ld=99)
    no(ERR_RANGE, "too large", ld=1 << 40)
    no(ERR_RANGE, "too large", probs_ld=1 << 40)
    no(ERR_RANGE, "R=", R=1 << 25)
    for name, word in (("x", "logits"), ("off", "offsets"), ("d", "drafts"), ("u", "u"), ("out", "out")):
        no(ERR_ARG, word + " is NULL", **{name: None})
    for name, word in (("x", "logits"), ("probs", "probs"), ("off", "offsets"), ("d", "drafts"), ("u", "u"),
                       ("temp", "temp"), ("out", "out"), ("p", "p_draft")):
        no(ERR_ALIGN, word, **{name: _up(b["beta"], 2)})
    no(ERR_ALIAS, "out overlaps drafts", out=b["v"])
    no(ERR_ALIAS, "p_draft overlaps probs", p=b["k"])
    no(ERR_ALIAS, "out overlaps p_draft", out=b["s_out"])
    need = lib.kda_accept_sampled_work_bytes(6, 3, 100)
    no(ERR_RANGE, "work_bytes", str(need), bytes=need - 1)
    no(ERR_ARG, "work is NULL", work=None)
    no(ERR_ALIGN, "work", work=_up(b["snap"], 8))
    assert _sampled(lib, b, R=0, x=None, d=None, u=None, probs=None, p=None, work=None, bytes=0) == OK
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 5000, 1)):
        assert lib.kda_accept_sampled_work_bytes(*bad) == -1


def test_python_binding_packs_the_caches_description():
    data = kda._pack_cache(1 << 40, 2, 3, 4, 5, 1 << 35, 7, 8, 9, 10)
    assert len(data) == ctypes.sizeof(_Cache)
    c = _Cache.from_buffer_copy(data)
    assert [getattr(c, n) for n, _ in _Cache._fields_] == [1 << 40, 2, 3, 4, 5, 1 << 35, 7, 8, 9, 10]


def test_python_binding_refuses_what_it_sees(lib):
    """Of tensors on the CPU; what needs a device is in the GPU tests."""
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_attn_rows(x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_cache_append(x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_accept_sampled(x, x, x, x, x)
    with pytest.raises(kda.KdaError):
        kda.attn_workspace(1, 0, 8, 1, device="cpu")
    with pytest.raises(kda.KdaError):
        kda.attn_workspace(1 << 32, 1, 8, 1, device="cpu")
    with pytest.raises(kda.KdaError):
        kda.accept_sampled_workspace(1, 1, 1 << 31, device="cpu")


def test_sampled_workspace_never_shrinks(lib):
    """One buffer of a loop's largest round serves every smaller one."""
    size = lib.kda_accept_sampled_work_bytes
    for B in (1, 15, 64, 4096):
        for V in (1, 7, 4096, 4097, 50001, 150000, 300007, 1 << 20, 1 << 30):
            last = 0
            for R in range(1, 4200, 1 if V == 150000 else 37):
                n = size(R, B, V)
                assert n >= last > -1
                last = n
            # what a call itself lays out, part by part of its rows: min(ceil(2048 / R), 64, whole parts of 4096 f32 logits)
            for R in (1, 2, 3, 31, 32, 33, 63, 511, 512, 2047, 2048, 2049, 4096):
                parts = min(-(-2048 // R), 64, -(-V // 4096))
                assert size(R, B, V) >= R * parts * 16
    for R in (1, 15, 511, 512, 5000):
        for B, V in ((1, 1000), (64, 150000)):
            assert size(R, B, V) <= min(size(R, B + 1, V), size(R, B, V + 1), size(R, B, 2 * V))


def test_attn_scales_that_leave_f32_in_base_2(lib, b):
    """2.4e38 log2(e) is an infinity in f32, and 0 times it a NaN."""
    for scale in (2.4e38, 3.4e38):
        _refused(lib, _attn(lib, b, R=0, q=None, o=None, scale=scale), ERR_RANGE, "scale")
    for scale in (1e-45, 1e-38, 1.0, 1.9e38):
        assert _attn(lib, b, R=0, q=None, o=None, scale=scale) == OK


class _Cpu:   # a device as the binding compares it: that of tensors on the CPU
    index = -1


def test_python_binding_refuses_a_cache_without_table_or_lengths(lib, b):
    k, v = torch.zeros(2, 4, 16, 2, 128).unbind()
    table = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="table"):
        kda._cache(k, v, None, torch.zeros(3, dtype=torch.int32), torch.float32, _Cpu)
    c, B, Hk = kda._cache(k, v, table, None, torch.float32, _Cpu)
    _refused(lib, lib.kda_cache_append(b["q"], 256, b["g"], 256, c, b["s_out"], 6, B, Hk, 0, None), ERR_ARG, "cache.lens is NULL")
    _refused(lib, lib.kda_attn_rows(b["q"], 512, c, b["s_out"], b["o"], 6, B, 4, Hk, 0.1, 0, 0, 0, b["snap"], 64 << 20, None),
             ERR_ARG, "cache.lens is NULL")


def test_python_binding_strides_of_one_page_row_or_head_are_free(lib, b):
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    one_page = torch.zeros(1, 16, 2, 128), torch.zeros(1, 2, 16, 2, 128)[:, 1]
    one_row = torch.zeros(4, 1, 2, 128), torch.zeros(4, 2, 1, 128).transpose(1, 2)
    one_head = torch.zeros(4, 16, 1, 128), torch.zeros(4, 1, 16, 128).transpose(1, 2)
    for k, v in (one_page, one_row, one_head):
        assert k.stride() != v.stride()
        for x, y in ((k, v), (v, k)):
            c = kda._cache(x, y, table, lens, torch.float32, _Cpu)[0]
            assert len(c) == ctypes.sizeof(_Cache)
    with pytest.raises(ValueError, match="same shape and strides"):
        kda._cache(torch.zeros(4, 16, 2, 128), torch.zeros(4, 2, 16, 128).transpose(1, 2), table, lens, torch.float32, _Cpu)


def test_python_binding_refuses_more_sequences_than_a_c_int_counts(lib):
    k, v = torch.zeros(2, 4, 16, 2, 128).unbind()
    with pytest.raises(kda.KdaError, match="32 bits"):
        kda._cache(k, v, torch.zeros(1 << 32, 0, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.float32, _Cpu)
