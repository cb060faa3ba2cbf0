"""Edges of shared attention's groups and own parts, and far positions of the append with a rotation.

Bounds as in tests/test_gpu_kv_shared.py; the rotation is held to equality."""
import numpy as np
import pytest
import torch

from test_gpu_kv import DEV, Case, exact, q  # noqa: F401  (q is a fixture)
from test_gpu_kv_shared import GROUPS, Shared, check, ints, run
from test_gpu_rotary import equal
from test_gpu_rotary import run as turn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,dim", [("decode", 64), ("decode", 256), ("crowd", 128), ("crowd", 256), ("prompts", 128)])
def test_groups_of_no_request(q, name, dim):  # noqa: F811
    """Between the others, first and last, sharing something or nothing."""
    c = Shared(q, GROUPS[name], 2, dim, 16).fill().append_new()
    first, shared = [0], []
    for g, s in enumerate(c.shared.tolist()):
        first += [first[-1], int(c.first[g + 1])]
        shared += [17 * g, s]
    first, shared = ints(first + [first[-1]]), ints(shared + [5])
    qx, out, lse = run(c, 12, first=first, shared=shared)
    check(c, out, lse, *exact(c, qx, dim ** -0.5, 0, 12))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,tokens", [(1, 1), (2, 3), (8, 1)])
def test_own_parts_about_the_longest_that_are_not_cut(q, dim, kv, tokens):  # noqa: F811
    step = 16 if dim == 256 else 32
    own = [24 * step + d for d in (-1, 0, 1)] + [25 * step + d for d in (-1, 0, 1)] + [3, 60 * step]
    for s in (64, 64 + step // 2):                                  # a prefix that ends at a step's end, and inside one
        c = Shared(q, [(s, [(n, min(n, tokens)) for n in own])], kv, dim, 64, seed=s).fill().append_new()
        qx, out, lse = run(c, 4 * kv)
        check(c, out, lse, *exact(c, qx, dim ** -0.5, 0, 4 * kv))
    q.q4nx_check(device=DEV)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,new", [([131072, 70001, 5000], [1, 3, 2]), ([131072, 70001], [900, 733])])
def test_rotation_far_out(q, lens, new, interleaved):  # noqa: F811
    equal(turn(q, Case(q, lens, new, 4, 64, 64), 8, 64, interleaved))
    q.q4nx_check(device=DEV)
