"""CPU checks of the room that the block operators need: the measured cases' own workspaces are
enough for every shape that they draw."""
import ctypes as C
import os
import random
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "perf"))
import more_operators as cases  # noqa: E402


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _draws(n):
    rng = random.Random(11)
    return cases.listed() + [cases.draw(rng) for _ in range(n)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are nobody's: only where nothing can be launched")
def test_the_cases_workspaces_are_enough(gs):
    """The calls of the cases' file, with addresses alone: they get as far as the GPU that is
    not there, instead of being refused for their room."""
    L, seen = gs.lib(), 0
    base = 1 << 40
    at = lambda i: base + (i << 36)  # noqa: E731  (arrays of their own)
    for case in _draws(4000):
        T = case["tokens"]
        dtype = 0 if case["dtype"] == "bf16" else 1
        if case["op"] == "ffn":
            c, f, room = case["width"], case["hidden"], cases.ffn_room(case)
            assert gs.gs_ffn_workspace_bytes(T, c, f, case["dir"] == "bwd") <= room, case
            continue
        if case["dir"] == "step":
            continue
        hq, hk, D, E, G = (case[n] for n in ("q_heads", "k_heads", "dim", "vdim", "groups"))
        row = hq * D + hk * D + hk * E  # one projection's
        a = gs.net._ATTN.pack(T, hq, hk, D, E, G, dtype, 1.0, at(8), at(9) if G > 1 else 0, at(10) if case["state"] else 0)
        q, k, v = (at(0), row, D), (at(0) + 2 * hq * D, row, D), (at(0) + 2 * (hq + hk) * D, row, E)
        out = (at(1), hq * E, E)
        room, states = cases.attn_room(case), at(11) if case["state"] else None
        if case["dir"] == "fwd":
            r = L.gs_linear_attn_fwd(a, gs.net._ATTN_HEADS4.pack(*q, *k, *v, *out), states, at(12), room, None)
        else:
            grads = [(p + at(2) - at(0), t, h) for p, t, h in (q, k, v)]
            r = L.gs_linear_attn_bwd(a, gs.net._ATTN_HEADS7.pack(*q, *k, *v, *out, *[x for g in grads for x in g]),
                                     states, states, at(12), room, None)
            seen += hq > hk and max(D, E) <= 64
        assert r == gs.GS_ERR_CUDA, (case, r)
    assert seen > 100


def test_rooms_that_are_asked_for(gs):
    """What is asked for grows no faster than two states for each 64 tokens and one more a
    group, but for copied rows, a quarter of the shared heads' gradients and two segments of
    them; less of it with fewer tokens' worth is refused only below two segments."""
    for T, H, K, D, E, G in [(32640, 16, 4, 64, 64, 1), (8160, 16, 4, 64, 64, 4), (2000, 16, 2, 64, 64, 1),
                             (1072, 4, 2, 16, 64, 1), (5003, 8, 4, 72, 41, 7), (9000, 8, 2, 128, 128, 1)]:
        d = 64 if max(D, E) <= 64 else 128
        up = lambda n: 64 if n <= 64 else 128  # noqa: E731
        states = 8 * (T // 64 + G) * H * d * d
        rows = 2 * T * (H + K) * (-(-D // 8) * 8 + -(-E // 8) * 8)
        part = 4 * H * (up(D) + up(E)) * (T // 4 + 1 + 2 * 2048)
        one = 8 * (T // 128 + G) * H * up(D) * up(E)
        assert gs.gs_linear_attn_workspace_bytes(T, H, K, D, E, G) <= max(states, one + rows + part) + 4096
