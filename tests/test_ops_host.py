"""The prompt, single-token and log-probability entry points refuse bad arguments on the host,
before anything is enqueued, and say what is wrong.

Every call below is one that validation must refuse (or that has nothing to enqueue).  Without a
GPU the pointers are aligned integers that validation never dereferences; with one they are
device buffers large enough for every shape used.
"""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_rows_amd as kda
from tests.test_abi_host import Bufs, ERR_ALIAS, ERR_ALIGN, ERR_ARG, ERR_RANGE, OK, _header_constant


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.lib_path()):
        from gated_delta_rule_rows_amd import build
        build.build()
    return kda.load()


@pytest.fixture(scope="module")
def b():
    return Bufs()


def _up(p, n):
    return ctypes.c_void_p(p.value + n)


def _prompt(lib, b, **kw):
    a = dict(s=b["ptrs"], off=b["s_in"], q=b["q"], k=b["k"], v=b["v"], g=b["g"], beta=b["beta"], o=b["o"],
             R=40, B=3, H=2, dt=0, work=b["snap"], bytes=32 << 20)
    a.update(kw)
    return lib.kda_prompt(a["s"], a["off"], a["q"], a["k"], a["v"], a["g"], a["beta"], a["o"], a["R"],
                          a["B"], a["H"], a["dt"], a["work"], a["bytes"], None)


def _linear(lib, b, **kw):
    a = dict(s=b["ptrs"], off=b["s_in"], q=b["q"], k=b["k"], v=b["v"], g=b["g"], o=b["o"],
             R=40, B=3, Hk=2, H=4, dt=0, work=b["snap"], bytes=32 << 20)
    a.update(kw)
    return lib.kda_linear_prompt(a["s"], a["off"], a["q"], a["k"], a["v"], a["g"], a["o"], a["R"], a["B"],
                                 a["Hk"], a["H"], a["dt"], a["work"], a["bytes"], None)


def _step(lib, b, **kw):
    a = dict(s=b["ptrs"], q=b["q"], k=b["k"], v=b["v"], g=b["g"], o=b["o"], L=2, B=3, Hk=2, H=4, dt=0)
    a.update(kw)
    return lib.kda_linear_step(a["s"], a["q"], a["k"], a["v"], a["g"], a["o"], a["L"], a["B"], a["Hk"],
                               a["H"], a["dt"], None)


def _logprobs(lib, b, **kw):
    a = dict(x=b["q"], t=3, V=100, ld=100, dt=0, tok=b["k"], n=5, lp=b["v"], ent=b["g"], ids=b["beta"],
             top=b["o"], work=b["snap"], bytes=32 << 20)
    a.update(kw)
    return lib.kda_logprobs(a["x"], a["t"], a["V"], a["ld"], a["dt"], a["tok"], a["n"], a["lp"], a["ent"],
                            a["ids"], a["top"], a["work"], a["bytes"], None)


def _refused(lib, rc, want, *words):
    said = lib.kda_last_error().decode()
    assert rc == want, said
    for w in words:
        assert w in said, said


def test_limits_match_the_header():
    assert _header_constant("KDA_TOP_MAX") == kda.TOP_MAX == 32


@pytest.mark.parametrize("call", [_prompt, _linear])
def test_prompt_refusals(lib, b, call):
    def no(want, *words, **kw):
        _refused(lib, call(lib, b, **kw), want, *words)

    no(ERR_ARG, "in_dtype", dt=2)
    no(ERR_RANGE, "R=-1", R=-1)
    no(ERR_RANGE, "R=", R=_header_constant("KDA_PROMPT_ROWS_MAX") + 1)
    no(ERR_RANGE, "B=0", B=0)
    no(ERR_RANGE, "B=", B=_header_constant("KDA_PROMPT_SEQS_MAX") + 1)
    no(ERR_RANGE, "H=0", H=0)
    no(ERR_RANGE, "H=", H=65536)
    no(ERR_RANGE, "R*H", R=1 << 28, H=65532)
    for name in ("s", "off", "q", "k", "v", "g"):
        no(ERR_ARG, "NULL", **{name: None})
    for name, step in (("s", 4), ("off", 2), ("q", 4), ("k", 8), ("v", 2), ("o", 4), ("g", 2)):
        have = {"s": "ptrs", "off": "s_in"}.get(name, name)
        no(ERR_ALIGN, "aligned", **{name: _up(b[have], step)})
    no(ERR_ALIAS, "o overlaps q", o=b["q"])
    no(ERR_ALIAS, "o overlaps v", o=_up(b["v"], 16))
    no(ERR_ALIAS, "o overlaps s_ptrs", o=b["ptrs"])
    no(ERR_ALIAS, "o overlaps offsets", o=b["s_in"])


def test_prompt_own_refusals(lib, b):
    _refused(lib, _prompt(lib, b, beta=None), ERR_ARG, "beta is NULL")
    _refused(lib, _prompt(lib, b, beta=_up(b["beta"], 2)), ERR_ALIGN, "beta")
    _refused(lib, _linear(lib, b, Hk=0), ERR_RANGE, "Hk=0")
    _refused(lib, _linear(lib, b, Hk=3), ERR_RANGE, "divide H=4")
    _refused(lib, _linear(lib, b, Hk=8), ERR_RANGE, "Hk=8")


@pytest.mark.parametrize("call,space", [(_prompt, "kda_prompt_work_bytes"),
                                        (_linear, "kda_linear_prompt_work_bytes")])
def test_prompt_workspace(lib, b, call, space):
    H = 2 if call is _prompt else 4
    need = getattr(lib, space)(40, 3, H)
    assert need >= 0
    if need:
        _refused(lib, call(lib, b, bytes=need - 1), ERR_RANGE, "work_bytes", str(need))
        _refused(lib, call(lib, b, work=None), ERR_ARG, "work is NULL")
        _refused(lib, call(lib, b, work=_up(b["snap"], 8)), ERR_ALIGN, "work")
        _refused(lib, call(lib, b, work=b["k"]), ERR_ALIAS, "work overlaps k")
        _refused(lib, call(lib, b, work=b["o"]), ERR_ALIAS, "o overlaps work")
    last = 0
    for R, B, heads in ((0, 1, 1), (1, 1, 1), (40, 1, 1), (40, 7, 1), (40, 7, 8), (100000, 7, 8), (100000, 400, 64)):
        n = getattr(lib, space)(R, B, heads)
        assert n >= last
        last = n
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 70000)):
        assert getattr(lib, space)(*bad) == -1


def test_prompt_without_rows_enqueues_nothing(lib, b):
    assert _prompt(lib, b, R=0, q=None, k=None, v=None, g=None, beta=None, o=None) == OK
    assert _linear(lib, b, R=0, q=None, k=None, v=None, g=None, o=None) == OK


def test_step_refusals(lib, b):
    def no(want, *words, **kw):
        _refused(lib, _step(lib, b, **kw), want, *words)

    no(ERR_ARG, "in_dtype", dt=-1)
    no(ERR_RANGE, "L=0", L=0)
    no(ERR_RANGE, "B=0", B=0)
    no(ERR_RANGE, "H=0", H=0)
    no(ERR_RANGE, "Hk=3", Hk=3)
    no(ERR_RANGE, "too large", L=1 << 16, B=1 << 16)
    no(ERR_RANGE, "too large", L=1 << 15, B=1 << 14)
    for name in ("s", "q", "k", "v", "g"):
        no(ERR_ARG, "NULL", **{name: None})
    no(ERR_ALIGN, "q", q=_up(b["q"], 8))
    no(ERR_ALIGN, "s_ptrs", s=_up(b["ptrs"], 4))
    no(ERR_ALIAS, "o overlaps k", o=b["k"])


def test_logprobs_refusals(lib, b):
    def no(want, *words, **kw):
        _refused(lib, _logprobs(lib, b, **kw), want, *words)

    no(ERR_ARG, "in_dtype", dt=5)
    no(ERR_RANGE, "t=0", t=0)
    no(ERR_RANGE, "V=0", V=0)
    no(ERR_RANGE, "outside 1..2^30", V=(1 << 30) + 1, ld=1 << 31)
    no(ERR_RANGE, "n_top=-1", n=-1)
    no(ERR_RANGE, "n_top=33", n=33)
    no(ERR_RANGE, "ld=99", ld=99)
    no(ERR_RANGE, "too large", ld=(1 << 40) // 3 + 1)
    no(ERR_ARG, "go together", tok=None)
    no(ERR_ARG, "go together", lp=None)
    no(ERR_ARG, "nothing", tok=None, lp=None, ent=None, n=0)
    no(ERR_ARG, "logits is NULL", x=None)
    no(ERR_ARG, "top_ids is NULL", ids=None)
    no(ERR_ARG, "top_lp is NULL", top=None)
    no(ERR_ALIGN, "logits", x=_up(b["q"], 2))
    no(ERR_ALIGN, "tokens", tok=_up(b["k"], 1))
    no(ERR_ALIGN, "lp", lp=_up(b["v"], 2))
    no(ERR_ALIAS, "lp overlaps logits", lp=b["q"])
    no(ERR_ALIAS, "top_ids overlaps tokens", ids=b["k"])
    no(ERR_ALIAS, "lp overlaps entropy", ent=b["v"])
    need = lib.kda_logprobs_work_bytes(3, 100, 5)
    if need:
        no(ERR_RANGE, "work_bytes", bytes=need - 1)
        no(ERR_ARG, "work is NULL", work=None)
        no(ERR_ALIAS, "work overlaps logits", work=b["q"])
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, -1), (1, 1, 33)):
        assert lib.kda_logprobs_work_bytes(*bad) == -1


def test_python_refuses_host_tensors():
    x = torch.zeros(2, 1, 128)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_prompt(torch.zeros(1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), x, x, x, x, x[..., 0])
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_linear_prompt(torch.zeros(1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), x, x, x, x[..., 0])
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_linear_step(torch.zeros(2, dtype=torch.int64), x[None], x[None], x[None], x[None, ..., 0])
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_logprobs(torch.zeros(2, 5))
    with pytest.raises(kda.KdaError, match="H=0"):
        kda.prompt_workspace(1, 1, 0)
    with pytest.raises(kda.KdaError, match="n_top"):
        kda.logprobs_workspace(1, 1, 40)


@pytest.mark.gpu
def test_python_refusals_on_device_tensors():
    R, B, Hk, H = 6, 2, 1, 2
    d = dict(device="cuda")
    s, off = torch.zeros(B, dtype=torch.int64, **d), torch.zeros(B + 1, dtype=torch.int32, **d)
    x, key = torch.zeros(R, H, 128, **d), torch.zeros(R, Hk, 128, **d)
    beta = torch.zeros(R, H, **d)
    work = kda.prompt_workspace(R, B, H)
    with pytest.raises(TypeError, match="offsets"):
        kda.kda_prompt(s, off.long(), x, x, x, x, beta, work=work)
    with pytest.raises(ValueError, match="offsets"):
        kda.kda_prompt(s, off[:-1], x, x, x, x, beta, work=work)
    with pytest.raises(TypeError, match="s_ptrs"):
        kda.kda_prompt(s.int(), off, x, x, x, x, beta, work=work)
    with pytest.raises(TypeError, match="q must be"):
        kda.kda_prompt(s, off, x.bfloat16(), x, x, x, beta, work=work)
    with pytest.raises(TypeError, match="v must be"):
        kda.kda_prompt(s, off, x, x, x.half(), x, beta, work=work)
    with pytest.raises(ValueError, match="beta"):
        kda.kda_prompt(s, off, x, x, x, x, beta[:, :1], work=work)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_prompt(s, off, torch.zeros(H, R, 128, **d).transpose(0, 1), x, x, x, beta, work=work)
    with pytest.raises(ValueError, match="g is on"):
        kda.kda_prompt(s, off, x, x, x, x.cpu(), beta, work=work)
    with pytest.raises(ValueError, match="o has shape"):
        kda.kda_prompt(s, off, x, x, x, x, beta, o=x[:3], work=work)
    with pytest.raises(kda.KdaError, match="divide"):
        kda.kda_linear_prompt(s, off, torch.zeros(R, 3, 128, **d), torch.zeros(R, 3, 128, **d), x, beta,
                              work=kda.linear_workspace(R, B, H))
    with pytest.raises(TypeError, match="g must be"):
        kda.kda_linear_prompt(s, off, key.bfloat16(), key.bfloat16(), x.bfloat16(), beta.bfloat16(),
                              work=kda.linear_workspace(R, B, H))
    with pytest.raises(ValueError, match="work"):
        kda.kda_linear_prompt(s, off, key, key, x, beta, work=torch.zeros(64, **d))
    with pytest.raises(ValueError, match="s_ptrs"):
        kda.kda_linear_step(s[:1], key[None], key[None], x[None], beta[None])
    logits = torch.zeros(4, 50, **d)
    tok, lp = torch.zeros(4, dtype=torch.int32, **d), torch.zeros(4, **d)
    w = kda.logprobs_workspace(4, 50, 3)
    with pytest.raises(TypeError, match="tokens"):
        kda.kda_logprobs(logits, tok.long(), lp, work=w)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        kda.kda_logprobs(torch.zeros(50, 4, **d).t(), tok, lp, work=w)
    with pytest.raises(ValueError, match="lp has shape"):
        kda.kda_logprobs(logits, tok, lp[:2], work=w)
    with pytest.raises(ValueError, match="go together"):
        kda.kda_logprobs(logits, top_lp=torch.zeros(4, 3, **d), work=w)
    with pytest.raises(kda.KdaError, match="rows would overlap"):
        kda.kda_logprobs(torch.zeros(60, **d).as_strided((4, 50), (3, 1)), tok, lp, work=w)


def test_grids_beyond_the_launch_limit_are_refused(lib, b):
    """A grid holds fewer than 2^32 threads; what would need more is refused before any launch."""
    for call, space in ((_prompt, lib.kda_prompt_work_bytes), (_linear, lib.kda_linear_prompt_work_bytes)):
        _refused(lib, call(lib, b, B=4096, H=257, Hk=257) if call is _linear else call(lib, b, B=4096, H=257),
                 ERR_RANGE, "B*H")
        _refused(lib, call(lib, b, R=1 << 28, H=65) if call is _prompt else call(lib, b, R=1 << 28, H=65, Hk=65),
                 ERR_RANGE, "R*H")
        assert space(40, 4096, 257) == -1
        assert space(40, 4096, 256) >= 0
        assert space(1 << 28, 1, 65) == -1
        assert space(1 << 28, 1, 64) > 0
    _refused(lib, _step(lib, b, L=1 << 10, B=1 << 12), ERR_RANGE, "L*B*H")      # 4 heads: 2^24
    _refused(lib, _logprobs(lib, b, t=1 << 26), ERR_RANGE, "t=67108864")
    assert lib.kda_logprobs_work_bytes(1 << 26, 1, 0) == -1
    assert lib.kda_logprobs_work_bytes((1 << 26) - 1, 1, 0) == 0


def test_linear_workspace_is_for_long_sequences_only(lib):
    """Part states take room for at most two parts of 512 rows a 512 rows, however many sequences
    there are: a batch of short prompts needs no more than one long one."""
    space, place = lib.kda_linear_prompt_work_bytes, 128 * 128 * 4 + 8
    for R, B, H in ((513, 4096, 256), (600, 64, 64), (4096, 256, 64), (8192, 256, 64), (100000, 4096, 64)):
        assert space(R, B, H) <= max(2 * R // 512 * H, 1) * place, (R, B, H)
        assert space(R, B, H) <= max(R * H // 2048, 2048) * place, (R, B, H)
    assert space(4096, 1, 64) == 9 * 64 * place
    # it never shrinks as a count grows, and holds what every smaller call needs
    counts = [(R, B, H) for R in (1, 512, 513, 1024, 5000, 70000, 1 << 20) for B in (1, 2, 9, 300, 4096)
              for H in (1, 3, 16, 64, 256)]
    for R, B, H in counts:
        n = space(R, B, H)
        for more in ((R + 1, B, H), (2 * R, B, H), (R, B + 1, H), (R, B, H + 1), (R, B, 2 * H)):
            if max(more[0] * more[2], 1) <= 1 << 34 and more[1] <= 4096 and more[1] * more[2] <= 1 << 20:
                assert space(*more) >= n, (R, B, H, more)


@pytest.mark.parametrize("call", [_prompt, _linear])
def test_prompt_without_rows_needs_no_workspace(lib, b, call):
    none = dict(R=0, q=None, k=None, v=None, g=None, o=None, work=None, bytes=0)
    if call is _prompt:
        none["beta"] = None
    assert call(lib, b, **none) == OK
    assert lib.kda_prompt_work_bytes(0, 4096, 64) == lib.kda_linear_prompt_work_bytes(0, 4096, 64) == 0


@pytest.mark.parametrize("space", [kda.prompt_workspace, kda.linear_workspace, kda.logprobs_workspace])
def test_counts_past_32_bits_are_refused(space):
    for at in range(3):
        counts = [1, 1, 1]
        counts[at] = 2 ** 32 + 1                   # 1, if it wrapped
        with pytest.raises(kda.KdaError, match="32 bits"):
            space(*counts, device="cpu")


@pytest.mark.gpu
def test_logits_past_32_bits_are_refused():
    lp, ent = torch.zeros(1, device="cuda"), torch.full((1,), 7.0, device="cuda")
    tok = torch.zeros(1, dtype=torch.int32, device="cuda")
    logits = torch.empty(1, 2 ** 32 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kda.KdaError, match="32 bits"):
        kda.kda_logprobs(logits, tok, lp, ent)
    assert float(ent) == 7.0
    with pytest.raises(kda.KdaError, match="outside"):
        kda.kda_logprobs(logits[:, :2 ** 30 + 1].contiguous(), tok, lp, ent)
