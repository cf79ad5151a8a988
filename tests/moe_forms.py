"""The rule by which the MoE layer picks its kernels' forms, restated from its
description, and layers of sizes that reach every form.

A form is (projection, n-tiles of 8 rows a segment holds at most, 16-row weight
tiles of a unit):
  n-tiles       twice the mean rows of an expert under an even choice, at most the
                tokens, and at most what fits beside two stages of the weight ring
  weight tiles  as many as leave a CTA three units or more
and the down projection also adds the rows up ("fused down") for up to 16 tokens,
two n-tiles and three units a CTA.
"""

STAGE_BYTES, SHARED_BYTES = 32768, 232448
SMS = 148


def _share(rows, E, n_out, outs, sms):
    """Units of a CTA's equal share when a unit has `outs` outputs."""
    return -(-min(rows, E) * -(-n_out // outs) // sms)


def _tiles(T, topk, E, K, n_out, halves, sms):
    rows = T * topk
    pitch = -(-K // 128) * 256 + 16
    other = 2 * STAGE_BYTES + 8 * 8 * 512 + (3 * 64 + 8) * 4 + (2 * 6 + 5) * 8 + 8 * rows + 4 * (E + 4)
    fit = (SHARED_BYTES - other) // pitch // 8 * 8
    n = min(-(-2 * rows // E), T, fit)
    nt = 1 if n <= 8 else 2 if n <= 16 else 4 if n <= 32 or halves == 2 else 8
    mt = 4 if _share(rows, E, n_out, 64 // halves, sms) >= 3 else \
        2 if _share(rows, E, n_out, 32 // halves, sms) >= 3 else halves
    if fit < 8 or nt == 4:
        mt = min(mt, 2)
    return nt, 1 if nt == 8 else mt


def forms(T, E, topk, K, F, N, gated, sms=SMS):
    """The two kernel forms of a layer: up and down projection."""
    up = _tiles(T, topk, E, K, F, 2 if gated else 1, sms)
    down = _tiles(T, topk, E, F, N, 1, sms)
    fused = T <= 16 and down[0] <= 2 and _share(T * topk, E, N, 16 * down[1], sms) <= 3
    return ("gated up" if gated else "up",) + up, ("fused down" if fused else "down",) + down


REACHABLE = {(kind, nt, mt) for kind in ("up", "down")
             for nt, mt in ((1, 1), (1, 2), (1, 4), (2, 1), (2, 2), (2, 4), (4, 1), (4, 2), (8, 1))} \
    | {("fused down", nt, mt) for nt in (1, 2) for mt in (1, 2, 4)} \
    | {("gated up", nt, mt) for nt, mt in ((1, 2), (1, 4), (2, 2), (2, 4), (4, 2))}

# (T, E, topk, K, F, N, gated)
LAYERS = [
    (1, 1, 1, 272, 144, 16, False), (9, 1, 1, 1040, 272, 48, False), (19, 1, 1, 528, 272, 40, True),
    (35, 1, 1, 528, 272, 40, False), (21, 8, 1, 272, 144, 80, True), (17, 4, 1, 528, 208, 40, True),
    (37, 214, 7, 272, 48, 48, False), (31, 15, 4, 272, 80, 624, False), (31, 156, 7, 144, 48, 80, True),
    (61, 112, 8, 272, 96, 112, False), (107, 154, 6, 64, 48, 168, True), (16, 63, 4, 48, 288, 216, False),
    (1, 3, 3, 272, 272, 6408, True), (9, 8, 5, 96, 528, 1280, False), (13, 16, 5, 64, 272, 1600, False),
    (43, 21, 4, 272, 464, 16, False), (85, 104, 6, 208, 144, 32, False),
]
