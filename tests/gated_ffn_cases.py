"""Sizes of the dense gated block that between them take every kernel its dispatch knows."""
import compressed_mixture_experts_amd as bm

# (tokens, d, ff)
SHAPES = [
    (126, 8, 96), (192, 120, 80), (512, 8, 8), (128, 1560, 3024), (540, 384, 5280), (75, 3848, 4288), (1312, 2576, 752), (3328, 2848, 64),
    (3654, 1616, 320), (2368, 2184, 432), (3165, 1288, 2944), (9090, 8, 3968), (12448, 3560, 264), (18176, 8, 7816), (17904, 136, 2088),
    (19015, 168, 8), (19067, 432, 200),
]


def kernels(tokens, d, ff):
    """What a training step of this size launches: product, tile form, whole or in shares (or
    which of them a joint launch has), and whether its depth ends inside a step."""
    p = bm.dbg_gated_ffn_plan(tokens, d, ff)

    def odd(depth, form, turned):
        return depth % (32 if turned and form == 3 else 64) != 0

    out = {("grad", p["grad"], odd(d, p["grad"], True))}
    if not p["few"]:
        out |= {("gate", p["gate"], odd(d, p["gate"], False)), ("y", p["y"], p["y_shares"] > 1, odd(ff, p["y"], False))}
    for name, depth, form, shares in zip(("dx", "dw", "dw"), (2 * ff, tokens, tokens), p["last"], p["last_shares"]):
        how = ("joint", bool(p["joint_parts"])) if p["joint"] else shares > 1
        out.add((name, form, how, odd(depth, form, True)))
    return out
