"""The two warps of a row's 128 columns in the 8-bit gated projection exchange their maxima through barriers of one
arrival.  Every order in which their steps can run is walked, with the barriers and parities of the source."""
import re
from pathlib import Path

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests import ffn_cases as fc
from tests.ssm_cases import gen

SOURCE = Path(binding.__file__).parent / "csrc" / "ida_gemm.cuh"


def stuck(arrive_on, wait_on, parity, tiles):
    """Whether some order of both warps' steps ends with one that waits for ever.  A warp's steps: arrive on the other's
    barrier arrive_on(n), wait on its own wait_on(n) until the phase of that parity is over."""
    todo, seen = [((0, 0), (0, 0, 0, 0))], set()  # steps done by either warp; phases of its two barriers, twice
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        steps, phases = state
        moved = False
        for w in (0, 1):
            n, waits = divmod(steps[w], 2)
            if n == tiles:
                continue
            after = list(phases)
            if not waits:
                after[2 * (1 - w) + arrive_on(n)] += 1
            elif phases[2 * w + wait_on(n)] & 1 == parity(n):
                continue
            moved = True
            todo.append((tuple(s + (i == w) for i, s in enumerate(steps)), tuple(after)))
        if not moved and min(steps) < 2 * tiles:
            return True
    return False


def test_no_order_of_steps_is_stuck():
    text = SOURCE.read_text().split("bool epi_gate_e4m3(")[1]
    arrive = re.search(r"arrive_local\(w\.in \+ other \* 2(?: \+ \((.*?)\))?\);", text)
    wait = re.search(r"pair_wait\(w\.in(?: \+ \((.*?)\))?, (.*?), g\.err\)", text)
    assert arrive and wait
    of = lambda expr: eval(f"lambda n: {expr or 0}")  # noqa: E731  (n, whole numbers, >> and &: the same in both languages)
    assert not stuck(of(arrive[1]), of(wait[1]), of(wait[2]), 7)


def test_one_barrier_is_stuck_in_some_order():
    assert stuck(lambda n: 0, lambda n: 0, lambda n: n & 1, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 128, 256, 400])
def test_many_tiles_of_short_contractions(D):
    """Contractions of one block and more, some thirty tiles to a pair of SMs: rows at the end as a call of their own has them."""
    T, F = 256 * 500, 640
    q, s = binding.ida_quant_e4m3(torch.randn(T, D, generator=gen(D)).cuda())
    w = [t.cuda() for i in (1, 2) for t in fc.quantised(torch.randn(F, D, generator=gen(D + i)), 128)]
    h, hs = binding.ida_glu_e4m3(q, s, *w)
    for at in (0, 256 * 123, T - 512):
        part, ps = binding.ida_glu_e4m3(q[at:at + 512].contiguous(), s[at:at + 512].contiguous(), *w)
        assert torch.equal(h[at:at + 512].view(torch.uint8), part.view(torch.uint8)) and torch.equal(hs[at:at + 512], ps)
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
