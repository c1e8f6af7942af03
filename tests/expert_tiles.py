"""Sizes at which the experts' products take their larger tiles, and the tiles that sizes take.
With tests/test_gpu_expert_ffn.py's own list every product meets each of its tiles."""

import combine_top_id_amd as M
from combine_top_id_amd.moonep import PRODUCTS

ROW_TILES = {(256, 256, False), (256, 128, False), (128, 64, False), (128, 32, False)}
TILES = {"gate_up": ROW_TILES, "down": ROW_TILES, "g_gate_up": ROW_TILES, "g_rows": ROW_TILES,
         "g_weights": {(256, 256, False), (256, 256, True), (128, 128, False), (128, 64, False)}}

# No width is a whole number of tiles or of steps.
LARGE_CASES = [
    # R, E, K, S, slots, H, I, maxvio
    (2, 4, 2, 5000, 1, 1032, 1032, 0.6),     # 256x256 everywhere, two tiles and more to a workgroup
    (3, 21, 3, 571, 1, 1000, 680, 3.0),      # 256x128, then 256x256 for gate and up; fallback pieces
    (4, 8, 2, 2000, 2, 1032, 712, 1.0),      # the two in turn, several tiles to a workgroup
    (2, 64, 8, 555, 1, 360, 1000, 2.0),      # 256x128 for many small groups; gradients past the caches
]


def tiles(R, E, K, S, slots, H, I):
    """Each product's tile at these sizes; no GPU is needed."""
    plan = M.Plan(M.moonep_query(R, E, K, S, slots), None, None)
    plan.desc.magic, plan.desc.dev, plan.desc.sz = 0x4D4F4E45, 256, plan.sz
    return {p: M.moonep_expert_tile(plan, H, I, p) for p in PRODUCTS}
