"""kda_logprobs over many rows: from 2048 on a wave has a row to itself, with one list and no others
to join it with.  And the size of its rounding errors, by their root mean square over the rows."""
import math

import pytest
import torch

from tests.test_gpu_logprobs import _call, _logits, _near, _want, NONE, inf

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
T = 2048


def _compare(got, want, V, threads, dtype):
    """A lane of a row's threads adds once for each 16-byte load, and its last and first loads may be
    single values; each load's own sum is 4 or 8 values deep and each exponential good to 2 places;
    64 lanes (and 4 waves) are joined by 8 more adds.  So log z is off by that many 2^-24 at most and
    a place of its own, x - m and the last subtraction round once each, and the entropy's second sum
    is off by as much relative to itself."""
    lp, ent, ids, top = got
    each = 16 // dtype.itemsize
    z = V / (each * threads) + 2 + each + 2 + 8 + 1
    _near(lp, want[0], 2.0 ** -24 * (z + 2 * want[0].abs().nan_to_num(0, 0, 0) + 2 * math.log(V + 1)))
    _near(ent, want[1], 2.0 ** -24 * (z * (1 + want[1].abs().nan_to_num(0) + math.log(V + 1))))
    if ids.shape[1]:
        assert torch.equal(ids.cpu(), want[2])
        _near(top, want[3], 2.0 ** -24 * (z + 2 * want[3].abs().nan_to_num(0, 0, 0) + 2 * math.log(V + 1)))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("t,V,n", [(T, 1, 1), (T, 3, 32), (T, 63, 0), (T, 64, 5), (T, 255, 32), (T + 1, 257, 1),
                                   (T, 512, 32), (T - 1, 513, 7), (T, 1025, 20), (T + 7, 2047, 32), (T, 4097, 3),
                                   (255, 700, 5), (256, 700, 5), (257, 1030, 32)])
def test_sizes(dtype, t, V, n):
    x, tok = _logits(t * V + n, t, V, DTYPES[dtype])
    _compare(_call(x.cuda(), tok.cuda(), n), _want(x, tok, n), V, 64 if t >= T else 256, DTYPES[dtype])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n", [1, 32])
def test_ties_take_the_lowest_index(dtype, n):
    V = 1201
    x, tok = _logits(1, T, V, DTYPES[dtype])
    x = x.round()
    x[0] = 2.0                                     # all equal: 0, 1, 2, ...
    x[1] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    x[T - 1] = -7.0
    _compare(_call(x.cuda(), tok.cuda(), n), _want(x, tok, n), V, 64, DTYPES[dtype])


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
def test_sorted_rows(order):
    V = 2011
    x = torch.linspace(-40, 10, V).expand(T, V).clone()
    if order == "falling":
        x = x.flip(1).contiguous()
    if order == "late":
        x = torch.full((T, V), -5.0)
        x[:, -40:] = torch.arange(40).float()
    tok = torch.full((T,), V - 1, dtype=torch.int32)
    _compare(_call(x.cuda(), tok.cuda(), 32), _want(x, tok, 32), V, 64, torch.float32)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [70, 1500])
def test_special_rows(dtype, V):
    dt = DTYPES[dtype]
    x, tok = _logits(2, T, V, dt)
    low = torch.finfo(dt).min
    at = T - 14                                    # behind rows that are plain
    x[at] = -inf
    x[at + 1, 1:] = -inf
    x[at + 2, 10:] = -inf
    x[at + 3, V // 2] = math.nan
    x[at + 4, V - 1] = inf
    x[at + 5] = math.nan
    x[at + 6, 3:] = low
    x[at + 7] = low
    x[at + 8, 5], x[at + 8, 6] = torch.finfo(dt).max, low
    x[at + 9] = 0.0
    x[at + 10, ::2] = -inf
    x[at + 11, 0] = 80.0
    x[at + 12, V - 1], x[at + 12, 0] = inf, math.nan
    x[at + 13, V - 1] = 60.0
    tok[at + 1], tok[at + 2], tok[at + 6], tok[at + 8], tok[at + 10], tok[at + 11] = 5, 3, V - 1, 6, 0, 0
    tok[at + 9] = V
    tok[at + 13] = NONE
    _compare(_call(x.cuda(), tok.cuda(), 20), _want(x, tok, 20), V, 64, dt)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (8, 3), (0, 8), (4, 12)])
def test_row_strides_and_alignment(dtype, offset, pad):
    V, dt = 601, DTYPES[dtype]
    gen = torch.Generator().manual_seed(offset + pad)
    flat = torch.full((offset + T * (V + pad),), math.nan, dtype=dt)   # what lies between the rows must not count
    x = flat[offset:].view(T, V + pad)[:, :V]
    x.copy_(3 * torch.randn(T, V, generator=gen))
    x = flat.cuda()[offset:].view(T, V + pad)[:, :V]
    tok = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
    _compare(_call(x, tok.cuda(), 9), _want(x.cpu(), tok, 9), V, 64, dt)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("t", [15, 512, T])
def test_rounding_errors_of_a_large_vocabulary(dtype, t):
    """Logits of deviation 3 over 150,000 entries: log z about 3.4 and the sums' quotient about -4, an
    entropy of 7.4 and log probabilities about as large.  In 2^-24: the logarithm rounds by 3.4 x 0.6,
    the sums' quotient and product by 4 x 0.3 each, the last subtraction by 7.4 x 0.3: 3.4 together.  n
    adds to a lane's running sum of equal parts leave 0.41 sqrt(n / 3) of it, an eighth of that over 64
    lanes: with n = 586 loads, 0.72 of z, and 5 times that (z counts once, w by 4) in the entropy: 3.6.
    Root of the squares 5.0, or 0.67 of the entropy; twice that is allowed, and as much for the log
    probabilities, in which the sums count once."""
    V = 150000
    gen = torch.Generator(device="cuda").manual_seed(t)
    x = (3 * torch.randn(t, V, generator=gen, device="cuda")).to(DTYPES[dtype])
    tok = torch.randint(0, V, (t,), generator=gen, device="cuda", dtype=torch.int32)
    lp, ent, ids, top = _call(x, tok, 8)
    want_lp, want_ent, want_top = [], [], []
    for part, k in zip(x.split(128), tok.split(128)):
        y = part.double()
        y = y - y.max(1, keepdim=True).values
        y = y - y.exp().sum(1, keepdim=True).log()
        want_lp.append(y.gather(1, k.long()[:, None])[:, 0])
        want_ent.append(-(y.exp() * y).sum(1))
        want_top.append(torch.sort(y, dim=1, descending=True, stable=True).values[:, :8])
    for got, want in ((lp, want_lp), (ent, want_ent), (top, want_top)):
        want = torch.cat(want)
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 1.34 * 2.0 ** -24, err * 2 ** 24
