"""The block-FP8 product's choice of a tile and of pieces of the reduction, written anew for the tests: which sizes
run which kernel.  The figures of the model are read from the source, so that a changed one changes the choice here
too; the number of pieces is compared with the library's workspace sizes (test_block_plan.py)."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "mixture_experts_layer_router_amd", "csrc", "fp8_matmul.hip")
PIECES = (1, 2, 3, 4, 6, 8, 12, 16, 24)


def forms():
    """[(mb, nb, fit, stage, out)] of the tiles, times in fp32 as the library holds them."""
    body = re.search(r"constexpr Form kForms\[\] = \{(.*?)\};", open(SOURCE).read(), re.S).group(1)
    found = []
    for mb, nb, fit, stage, out in re.findall(r"\{(\d+), (\d+), (\d+), \{([^}]*)\}, ([\d.]+)f\}", body):
        found.append((int(mb), int(nb), int(fit), [float(np.float32(v.strip().rstrip("f"))) for v in stage.split(",")],
                      float(np.float32(out))))
    return found


FORMS = forms()


def up(a, b):
    return -(-a // b)


def plan(M, N, K):
    """(form, pieces): of those that fit, the one that the model gives the least time, the first of equal ones."""
    nkb, best = up(K, 128), None
    for f, (mb, nb, fit, stage, out) in enumerate(FORMS):
        tiles = up(M, mb * 64) * up(N, nb * 64)
        for want in PIECES:
            chunk = up(nkb, want)
            pieces = up(nkb, chunk)
            if pieces != want or (pieces > 1 and tiles * pieces > 1024):
                continue
            each = up(tiles * pieces, 256)  # units of a CU
            t = each // fit * stage[fit - 1] + (stage[each % fit - 1] if each % fit else 0.0)
            t = 4 + t * chunk + out * each + (2.5 + pieces * M * N * 8 / 5e6 if pieces > 1 else 0)
            if best is None or t < best[0]:
                best = (t, f, pieces)
    return best[1:]
