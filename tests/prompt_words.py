"""The words that the prompts' kernels take their operands apart into, in numpy, with the option of a
mistake, and the bound that tells them apart."""
import numpy as np

# Relative 2-norm error of outputs and states of plain prompts.  An output is a few products of at
# most 128 terms each: operands of 22 bits or more (rounded by 2^-23 at most, 0.6 x 2^-24 root mean
# square each, and the product that is left out as much), and a dozen roundings of running f32 sums
# by as much again.  Their squares add to under (8 x 2^-24)^2 with the decays' roundings; twice that.
BOUND = 2.0 ** -20


def bf16_words(x, n):
    """x (f32) as n words of 8 bits, cut off, highest first: three are x itself."""
    rest, words = x.astype(np.float32), []
    for _ in range(n):
        w = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        words.append(w.astype(np.float64))
        rest = rest - w
    return words


def f16_words(x, axis):
    """x scaled by a power of two for each row or column, as two f16 words; with the scales."""
    most = np.abs(x).max(axis=axis, keepdims=True)
    s = 2.0 ** (13 - np.floor(np.log2(most)))
    hi = (x * s).astype(np.float16)
    lo = (x * s - hi.astype(np.float64)).astype(np.float16)
    return [hi.astype(np.float64), lo.astype(np.float64)], s


def bf16_product(a, b, words_a, words_b, lost=()):
    """a . b over words, without the products (i, j) in lost and those whose places add to over 2."""
    wa, wb = bf16_words(a, words_a), bf16_words(b, words_b)
    out = 0.0
    for i in range(words_a):
        for j in range(words_b):
            if i + j <= 2 and (i, j) not in lost:
                out = out + wa[i] @ wb[j]
    return out


def f16_product(a, b, lost=()):
    wa, sa = f16_words(a.astype(np.float64), 1)
    wb, sb = f16_words(b.astype(np.float64), 0)
    out = 0.0
    for i, j in ((1, 0), (0, 1), (0, 0)):
        if (i, j) not in lost:
            out = out + wa[i] @ wb[j]
    return out / sa / sb
