"""The exchange of largest magnitudes between the two blocks of a gated 8-bit
tile: a model of its barriers run through every interleaving on the CPU, with
the number of barriers that the kernel declares; and the kernel on tiles whose
reductions are so short that one block can be a tile ahead of the other.

In the model a block has two threads: the one that publishes and one that may
be late.  A tile, as in the kernel: both meet, the first publishes to the other
block, both wait for the other block's publication and read its values, both
meet again.  Nothing else holds a block back, as with short reductions.
"""
import os
import re

import pytest
import torch

from combine_ep_prepare_gb300 import workloads as wl
from tests.test_experts_gpu import STEP, Step, ep  # noqa: F401
from tests.test_f8_products_gpu import act_bounds, columns, per_expert, rows8, same, weights8
from tests.test_f8_rows_gpu import F8

SOURCE = os.path.join(os.path.dirname(wl.__file__), "csrc", "ep_products_f8.cu")
TILES = 5
STEPS = ["meet", "publish", "wait", "read", "meet"]  # the second thread publishes nothing


def stuck_or_torn(buffers, barriers):
    """Every interleaving of TILES tiles: whether one ends with a thread that
    waits for ever, and whether one reads a buffer of another tile's values."""
    # A thread's place counts steps; per block: tile whose values lie in each
    # buffer, and how often each barrier's phase has ended.
    start = ((0,) * 4, ((-1,) * buffers,) * 2, ((0,) * barriers,) * 2)
    seen, todo, stuck, torn = {start}, [start], False, False
    while todo:
        place, data, phases = todo.pop()
        moved = False
        for who in range(4):
            block, other = who // 2, 1 - who // 2
            tile, step = divmod(place[who], len(STEPS))
            if tile == TILES:
                continue
            mate = place[who ^ 1]
            p, d, ph = list(place), [list(x) for x in data], [list(x) for x in phases]
            if STEPS[step] == "meet":
                if mate < place[who]:
                    continue  # the other thread is not there yet
            elif STEPS[step] == "publish" and who % 2 == 0:
                d[other][tile % buffers] = tile
                ph[other][tile % barriers] += 1
            elif STEPS[step] == "wait":
                if ph[block][tile % barriers] % 2 == tile // barriers % 2:
                    continue  # the phase at hand has the parity that is waited for
            elif STEPS[step] == "read":
                torn = torn or data[block][tile % buffers] != tile
            p[who] += 1
            moved = True
            state = (tuple(p), tuple(map(tuple, d)), tuple(map(tuple, ph)))
            if state not in seen:
                seen.add(state)
                todo.append(state)
        stuck = stuck or not moved and any(x < TILES * len(STEPS) for x in place)
    return stuck, torn


def test_model_finds_what_one_barrier_allows():
    assert stuck_or_torn(2, 1) == (True, False)
    assert stuck_or_torn(1, 1)[1]
    assert stuck_or_torn(2, 2) == (False, False)


def test_kernel_has_a_barrier_for_each_buffer():
    with open(SOURCE) as f:
        code = f.read()
    sizes = {m[0]: int(m[1]) for m in re.findall(r"constexpr int (\w+) = (\d+);", code)}
    count = lambda name: sizes.get(name) or int(name)  # noqa: E731
    buffers = count(re.search(r"float peer_max\[(\w+)\]\[kTileN\]", code)[1])
    halves = re.search(r"\bpeer_full\[(\w+)\](?:\[(\w+)\])?;", code)
    barriers = 1 if halves[2] is None else count(halves[1])
    assert stuck_or_torn(buffers, barriers) == (False, False)
    uses = re.findall(r"s\.peer_full((?:\[\w+\])+)", code)
    assert uses and all(u in ("[turn][half]", "[i][j]") for u in uses)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K,T,n_in,f", [(4, 1, 8192, 128, 2048), (3, 1, 6000, 16, 2048), (2, 1, 5000, 256, 2048), (64, 2, 128, 1024, 2048)])
def test_gated_tiles_of_short_reductions(ep, E, K, T, n_in, f):  # noqa: F811
    """Several tiles a pair: the 8-bit result against 64 bits, the same in every
    call, and no wait that gave up."""
    s = Step(ep, E, K, T, 1, "bf16", 60, p_mask=0.0)
    x, xs, xv = rows8(ep, s, n_in, 61)
    w, ws, wv = weights8(ep, E, 2 * f, n_in, 62)
    q, qs = torch.empty(s.R, f, dtype=F8, device="cuda"), torch.empty(s.R, columns(f), device="cuda")
    ep.ep_expert_gemm_f8_swiglu(s.h, x, xs, w, ws, act_q=q, act_scales=qs)
    want, mag = per_expert(s, xv, wv.transpose(1, 2), 2 * f)
    a, off = act_bounds(want, mag, f, n_in)
    live = s.live.cuda()
    m, off_m = a.abs().view(s.R, -1, 128).amax(2), off.view(s.R, -1, 128).amax(2)
    scale = qs[:, :f // 128].double()
    assert bool(((scale - m / 448).abs() <= (off_m + 4 * STEP * m) / 448 + 1e-30)[live].all())
    scale = scale.repeat_interleave(128, 1)
    assert bool(((q.double() * scale - a).abs() <= a.abs() * (2.0 ** -4 + 1e-6) + scale * 2.0 ** -10 + 1.1 * off)[live].all())
    for _ in range(50):
        q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
        ep.ep_expert_gemm_f8_swiglu(s.h, x, xs, w, ws, act_q=q2, act_scales=qs2)
        assert same(q2[:s.P], q[:s.P]) and same(qs2[:s.P], qs[:s.P])
    assert ep.ep_read_info(s.h)["status"] == 0
