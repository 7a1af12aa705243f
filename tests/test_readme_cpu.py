"""The README's other examples name what the binding has, with the settings
that they mean (no GPU)."""
import os
import re

from speculative_decode_tree_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TEXT = open(os.path.join(ROOT, "README.md")).read()


def test_the_target_models_rotation_does_not_scale():
    # 512 + 64 MLA models put YaRN's attention factor into the softmax scale: sine and cosine stay as they are.
    from speculative_decode_tree_gb300.build import build
    build()
    call = re.search(r"^rope = (B\.ddtree_rope_init\(.*?\))$", TEXT, re.M | re.S).group(1)
    rope = eval(call)
    assert rope.rot_dim == 64 and rope.interleaved == 1 and rope.mscale == 1.0


def test_bound_calls_are_the_ones_that_exist():
    have = {n for n in vars(B) if n.startswith("Bound")}
    assert have and set(re.findall(r"\bBound[A-Z]\w+", TEXT)) == have
