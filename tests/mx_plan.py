"""The rule by which a product with MXFP4 weights is streamed or goes in tiles, for tests that want a
certain form (no test functions).  It mirrors plan_mx_product; test_mx_plan.py holds it to the
library's workspace sizes, which depend on the form."""
from __future__ import annotations

import math
from dataclasses import dataclass

CUS = 256
PLANES = {"f32": 3, "h2": 2, "bf16": 1, "mx": 1}  # h2: the h of bf16 rows


def _up(a, b):
    return -(-a // b)


@dataclass
class Form:
    bm: int = 0          # 0: streamed
    cols: int = 0
    shared: bool = False  # tiles cut along K, their sums in the workspace
    rest: tuple | None = None  # (rows, columns) of the tiles of a last round
    plane_bytes: int = 0

    def __str__(self):
        if self.bm == 0:
            return "stream"
        return f"{self.bm}x{self.cols}" + (" shared" if self.shared else "") + (f" rest {self.rest[0]}x{self.rest[1]}" if self.rest else "")


def product(M, N, K, kind, glu=False) -> Form:
    if M <= 16:
        return Form()
    mats, planes, fp4 = 2 if glu else 1, PLANES[kind], kind == "mx"
    cols, S = 256 // mats, _up(K, 128)
    bm = 32 if M <= 32 else 64 if M <= 64 else 128
    col_tiles = _up(N, cols)
    if fp4 and M > 128:
        rows, wide = _up(M, 128), _up(N, 2 * cols)
        if _up(rows * wide, CUS) * (1.35 if glu else 1.7) < _up(rows * col_tiles, CUS):
            cols, col_tiles = 2 * cols, wide
    tiles = _up(M, bm) * col_tiles
    f = Form(bm, cols)
    units, sums_us = _up(S, 2) * _up(tiles, CUS), 0.0
    if tiles < CUS and S > 2:
        per = _up(S, 2)
        quota = max(2, _up(tiles * per, CUS))
        most = (per + quota - 2) // quota + 1
        unit_us = max(2.0 * bm * 256 * 256 * planes / (12e6 if fp4 else 5e6), 35e3 / 23e3)
        us = 2 * min(float(most), 1 + per / quota) * 4.0 * M * N * mats / 4e6
        if quota < per and (per - quota) * unit_us > 4 + us:
            f.shared, f.plane_bytes, units, sums_us = True, most * mats * M * N * 4, quota, us
    if M > 128 and tiles > CUS and tiles % CUS:
        full, narrow = tiles // CUS * CUS // _up(M, bm) * cols, 256 // mats
        wide = cols != narrow
        step_us = (0.92 if wide else 0.62) if fp4 else 1.5 * planes
        rounds = lambda b: math.ceil(math.ceil(M / b) * _up(N - full, narrow) / CUS)  # noqa: E731
        half = rounds(64) * (0.6 if not fp4 else (0.56 if glu else 0.49) if wide else (0.8 if glu else 0.72))
        other = rounds(128) * 0.69 if wide else 1
        if full > 0 and (1 - min(half, other)) * S * step_us > 4:
            f.rest = (64 if half < other else 128, narrow)
    if M <= 128:
        i = ("f32", "h2", "bf16", "mx").index(kind)
        start, own = (3.5, 3.5, 3, 2.7)[i], (0.5, 0.4, 0.2, 0.2)[i]
        step = ((0.21, 0.20, 0.14, 0.125), (0.35, 0.35, 0.27, 0.24))[glu][i]
        wgs = _up(N, 32) * _up(M, 16) / CUS
        stream_us = start + (math.ceil(wgs) + wgs) / 2 * (own + S * step)
        h = (32, 64, 128).index(bm)
        base, stage = (((8.5, 10.3, 12), (0.8, 1.5, 2.5)), ((6.8, 7.8, 7), (0.7, 0.8, 1)))[fp4]
        if stream_us < base[h] + (2.3 if kind == "f32" else 0) + units * planes * stage[h] + sums_us:
            return Form()
    return f


def _carve(parts):
    cursor = 0
    for n in parts:
        cursor = _up(cursor + n, 256) * 256
    return cursor


PIECES = {"f32": 6, "h2": 4, "bf16": 0, "mx": 0}  # bytes of a value's bf16 planes


def gemm_bytes(M, K, N, kind):
    f = product(M, N, K, kind)
    return max(_carve([PIECES[kind] * M * K, f.plane_bytes]) if f.bm else 0, 256)


def mlp(M, H, I, kind):
    """(gate and up's form, down's)."""
    return product(M, I, H, kind, True), product(M, H, I, "h2" if kind == "bf16" else kind)


def mlp_bytes(M, H, I, kind):
    gu, dn = mlp(M, H, I, kind)
    n = M * I
    h = [n // 2, n // 32] if kind == "mx" else [PIECES["h2" if kind == "bf16" else kind] * n if dn.bm else 4 * n]
    return max(_carve(h + [PIECES[kind] * M * H if gu.bm else 0, max(gu.plane_bytes, dn.plane_bytes)]), 256)
