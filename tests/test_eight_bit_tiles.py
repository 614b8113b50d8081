"""Which of the W8A8 product's seven tiles a call takes, on the host from the rule in the source, so
that the shapes which the GPU tests run through whole stages of each tile keep doing so."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_activation_quantized_amd", "csrc",
                      "mixllm_gemm8.hip")

# tile, tokens, channels, inputs: whole stages that fill the ring twice and a part of one, where channels
# and tokens fill their last tile or leave some of it
LOOPS = [("32x32", 4, 1000, 8208), ("32x32", 32, 4096, 2064), ("32x64", 33, 4100, 2080), ("32x64", 64, 5120, 1808),
         ("64x64", 65, 8192, 1040), ("64x64", 100, 8101, 1200), ("64x128", 256, 8192, 1040), ("64x128", 250, 8011, 1168),
         ("128x128", 1024, 4096, 1040), ("128x128", 1000, 4011, 2064), ("256x128", 2047, 4096, 1040),
         ("256x128", 2048, 4090, 912), ("256x256", 3900, 3601, 1040), ("256x256", 4096, 4096, 656)]
STRIDED = [("32x32", 20, 333, 2064), ("32x64", 64, 5001, 1808), ("64x64", 100, 8101, 1040), ("64x128", 250, 8011, 1040),
           ("128x128", 1000, 4011, 1040), ("256x128", 2000, 4090, 1040), ("256x256", 3900, 3601, 656)]


def rule():
    """(tokens, channels, us) of the kinds of tiles, and their (inputs of a stage, stages)."""
    with open(SOURCE) as f:
        text = f.read()
    kinds = [(int(m), int(n), float(us)) for m, n, us in re.findall(r"\{(\d+), (\d+), ([\d.]+)f\}", text)]
    ring = {f"{m}x{n}": (int(bk), int(st)) for m, n, bk, st in
            re.findall(r"using Tile\w+ = TileShape<(\d+), (\d+), \d+, \d+, \d+, (\d+), (\d+)>", text)}
    return kinds, ring


def picked(m, n, k):
    kinds, _ = rule()
    f = np.float32
    floor = (f(m) * f(k) + f(n) * f(k) + f(2) * f(m) * f(n)) / f(5.5e6)
    best = None
    for i, (tm, tn, us) in enumerate(kinds):
        if i and tm >= 2 * m:
            break
        tiles = -(-m // tm) * -(-n // tn)
        rounds = f((tiles + 255) // 256) * f(us) * f(k) / f(4096)
        cost = max(rounds, floor) + f(0.1) * rounds
        if best is None or cost < best[0]:
            best = cost, f"{tm}x{tn}"
    return best[1]


def test_the_rule_is_read():
    kinds, ring = rule()
    assert len(kinds) == 7 and [f"{m}x{n}" for m, n, _ in kinds] == ["32x32", "32x64", "64x64", "64x128", "128x128", "256x128", "256x256"]
    assert set(ring) == {f"{m}x{n}" for m, n, _ in kinds}
    assert picked(512, 4096, 4096) == "64x128" and picked(2047, 14336, 4096) == "256x256" and picked(4, 28672, 8192) == "32x32"


@pytest.mark.parametrize("shapes", [LOOPS, STRIDED], ids=["loops", "strided"])
def test_shapes_take_every_tile_through_its_stages(shapes):
    _, ring = rule()
    assert {t for t, _, _, _ in shapes} == set(ring)
    for tile, m, n, k in shapes:
        bk, st = ring[tile]
        assert picked(m, n, k) == tile, (tile, m, n, k, picked(m, n, k))
        assert k // bk >= 2 * st and k % bk, (tile, k)

