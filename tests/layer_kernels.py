"""Calls of the layer operators that reach every kernel of their products, with the kernel that each is to
reach: the tests on the CPU check that it does, those on the GPU check its results."""
from typing import NamedTuple


class Product(NamedTuple):
    """A call of linear8 or gated8.  `packed`: x comes in 8 bits; `dtype` is x's and y's."""
    gated: bool
    tokens: int
    rows: int
    cols: int
    dtype: str = "bf16"
    keep: bool = False
    pack: str | None = None
    x: str = "e4m3"
    w: str = "e4m3"
    packed: bool = False
    activation: str = "none"
    bias: bool = False
    residual: bool = False
    exact: bool = False


class Grad(NamedTuple):
    """A call of weight_grad8 (n = 0) or of input_grad8 for n layers.  fp32 gradients take part in three terms each, or
    without `exact` in two, fp16 ones in two."""
    n: int
    tokens: int
    rows: int
    cols: int
    dtype: str = "bf16"
    fmt: str = "e4m3"
    exact: bool = True


def products():
    """(tokens of a tile, codes widened to bf16, call): every tile over one block of 128 columns, over more than the
    loop's four, past the 56 whose scales are in shared memory at a time, and with a last block of one column."""
    got = []
    for gated in (False, True):
        half = 2 if gated else 1  # a tile holds 256 rows of weights, or 128 of either projection
        for n, (tt, wide, tokens, rows, dtype) in enumerate([
                (64, False, 700, 1300, "bf16"), (128, False, 2048, 2600, "bf16"), (256, False, 4100, 2600, "bf16"),
                (64, True, 60, 120000, "bf16"), (64, True, 50, 1300, "fp16"), (128, True, 300, 1030, "fp32")]):
            call = Product(gated, tokens, rows // half, 0, dtype)
            kept = rows < 5000  # (kept or packed with few tokens: the tile; neither: the tile only for many outputs)
            for m, cols in enumerate([100, 640, 1000, 7300] if kept else [1100, 1153]):
                got.append((tt, wide, call._replace(
                    cols=cols, keep=kept and m != 1, pack="e5m2" if kept and m == 1 else None, packed=m == 2,
                    dtype="fp16" if dtype == "bf16" and m % 2 else dtype, activation=("none", "silu", "gelu", "relu")[(m + n) % 4],
                    bias=not gated and m < 2, residual=not gated and m > 0)))
            for x, w in (("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")):
                got.append((tt, wide, call._replace(cols=900 if kept else 1153, x=x, w=w, keep=kept)))
        for n, cols in enumerate((900, 7300)):  # 8 and 16 bits of every product
            call = Product(gated, 700, 1300 // half, cols, ("bf16", "fp16")[n], True, ("e4m3", None)[n], activation="silu", exact=True)
            got += [(128, True, call), (64, True, call._replace(tokens=50))]
    return got


def few():
    """(blocks of 16 tokens, waves, call): few tokens, up to one chunk of the columns and past it."""
    got = []
    for gated in (False, True):
        for i, tokens in enumerate((1, 2, 4, 5, 16, 17, 32, 33, 64)):
            nt = 1 if tokens <= 16 else 2 if tokens <= 32 else 4
            for rows in (8192, 8203):
                for n, cols in enumerate((130, 1000, 2048, 2100)):
                    got.append((nt, 4, Product(gated, tokens, rows, cols, ("bf16", "fp16", "fp32", "bf16")[(n + i) % 4],
                                               activation=("silu", "none", "gelu")[n % 3], bias=not gated and n > 1,
                                               residual=not gated and n < 2)))
            for n, (x, w) in enumerate([("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")]):
                got.append((nt, 4, Product(gated, tokens, 8200, 2100, ("fp32", "fp16", "bf16")[(n + i) % 3], x=x, w=w)))
                got.append((nt, 8, Product(gated, tokens, 200, 4300, ("fp16", "bf16", "fp32")[(n + i) % 3], x=x, w=w)))
    return got


def gradients():
    """(rows of a tile, whether the sum is in parts, call): odd and even numbers of steps of 64, one to six pairs
    of matrices, rows of dy that are whole 16-byte pieces and others."""
    got = []
    for fmt in ("e4m3", "e5m2"):
        for tokens in (1, 64, 65, 192, 260):
            got.append((256, False, Grad(0, tokens, 3304, 3300, "bf16", fmt)))
        got += [(256, False, Grad(0, 200, 3301, 3300, "bf16", fmt)), (256, False, Grad(0, 130, 3301, 3309, "fp32", fmt)),
                (256, True, Grad(0, 4000, 2704, 900, "bf16", fmt)), (256, True, Grad(0, 4003, 2701, 897, "bf16", fmt)),
                (256, True, Grad(0, 2000, 2704, 900, "fp16", fmt)), (256, True, Grad(0, 1003, 2701, 900, "fp32", fmt)),
                (256, True, Grad(0, 2000, 2701, 900, "fp32", fmt, False))]
        for rows in (8, 64, 72, 192, 257):
            for n in (1, 2):
                got.append((256, False, Grad(n, 3301, rows, 3300, "bf16", fmt)))
        got += [(256, False, Grad(2, 3300, 130, 3301, "fp32", fmt)), (256, True, Grad(1, 2701, 4000, 900, "bf16", fmt)),
                (256, True, Grad(2, 2703, 2001, 897, "bf16", fmt)), (256, True, Grad(2, 2700, 1000, 900, "fp16", fmt)),
                (256, True, Grad(2, 2700, 500, 900, "fp32", fmt)), (256, True, Grad(2, 2701, 1000, 900, "fp32", fmt, False)),
                (128, False, Grad(0, 700, 1024, 2304, "bf16", fmt)), (128, True, Grad(2, 129, 2000, 300, "fp32", fmt))]
    return got
