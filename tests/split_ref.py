"""Keys and values of which every stretch of 32 counts: a score for each stretch, and the stretch's values 1 in one
channel and 0 in the others, so that a channel of the result is the weight of its stretches and a stretch that is lost,
or counted twice, is a tenth of its channel and more."""
import torch

D = 128
STRETCH = 32   # keys: half a tile of bf16 keys, a whole one of f32 keys


def keys_and_values(length, gen, even):
    """Scores of the keys (exact in bf16; even: all 0) and the values' channels, by position."""
    channel = torch.arange(length) // STRETCH % D
    scores = torch.randint(-96, 97, (D,), generator=gen).double() / 16      # -6 .. 6
    return torch.zeros(length).double() if even else scores[channel], channel


def result(scores, channel, factor, count):
    """The channels of a row that sees keys 0 .. len(scores) - 1, each counted count[j] times."""
    w = torch.exp((scores - scores.max()) * factor if factor > 0 else (scores - scores.min()) * factor) * count
    return torch.zeros(D, dtype=torch.float64).index_add_(0, channel, w) / w.sum()


def bound(keys, dt, even):
    """How far a channel may be off, of itself.  Every weight is positive and a channel adds the weights of its own
    keys alone.  Half steps of f32 (2^-24): 18 of a weight's exponent (log2(e) in f32 times up to 8.7, a difference of
    up to 17.4 in base 2) and 2 of its exponential, on both sides of the quotient; one a key of a channel and one a 16
    keys of the sum l (its chains take a tile of 32 or 64 keys in one addition, after 8 of 16 a lane); 40 of
    moves to a new maximum, of the join and of the quotient.  With even scores all weights are 1, and sums are exact.
    bf16 rounds the weights, unless they are 1, and the result."""
    steps = 4 if even else 40 + 40 + keys // D + 2 * STRETCH + keys // 16 + 10
    rel = steps * 2.0 ** -24
    if dt == torch.bfloat16:
        rel = rel + (0 if even else 2.0 ** -8)
        rel = rel + 2.0 ** -8 * (1 + rel)
    return rel


def off(got, want, rel):
    """Whether a channel is further off than its bound."""
    return bool(((got - want).abs() > rel * want).any())
