"""The layers of tests/moe_forms.py reach every form of the MoE layer's kernels,
and nothing reaches another one."""
import random

from moe_forms import LAYERS, REACHABLE, forms


def test_layers_reach_every_form():
    assert {f for layer in LAYERS for f in forms(*layer)} == REACHABLE


def test_no_other_form_is_reachable():
    r = random.Random(5)
    seen = set()
    for _ in range(60000):
        T, E, topk = int(2 ** r.uniform(0, 7.01)), int(2 ** r.uniform(0, 10.01)), r.randint(1, 8)
        K, F, N = 16 * int(2 ** r.uniform(0, 9.01)), 16 * int(2 ** r.uniform(0, 9.01)), 8 * int(2 ** r.uniform(0, 13.01))
        seen.update(forms(min(T, 128), min(E, 1024), topk, min(K, 8192), min(F, 8192), N, r.random() < 0.5))
    assert seen <= REACHABLE
