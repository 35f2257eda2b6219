"""kda_logprobs over many rows: from 2048 on a wave has a row to itself, with one list and no others
to join it with.  And the size of its rounding errors, by their root mean square over the rows."""
import pytest
import torch

from tests.test_gpu_logprobs import _call

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
T = 2048


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
