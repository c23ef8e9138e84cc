"""The example that runs the 8-bit operators together, with its own check against 64 bits."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "decode_8bit", os.path.join(ROOT, "examples", "decode_8bit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
def test_decode_example_against_64_bits():
    """Every output within its rounding and 2^-7 of what the probabilities weigh, the tiers'
    slots all used, and the pool as one request leaves it."""
    e = _example()
    worst, _, m = e.run(steps=5, check=True)
    assert worst <= 1.0
    assert int(m.slots[:e.R - 1].max()) > e.HOT            # resident rows were read
    assert bool((m.slots[:e.R - 1] == e.HOT).any())        # and the newest
    refs, tables = m.pool.refs.cpu(), m.pool.tables.cpu()
    held = tables[1][tables[1] >= 0]
    assert held.tolist() == sorted(held.tolist()) and len(held) == e.RESIDENT
    assert sorted(held.tolist()) == list(range(e.RESIDENT))   # compacted to the front
    assert torch.equal(refs, torch.cat([torch.ones(e.RESIDENT, dtype=torch.int32),
                                        torch.zeros(e.PAGES - e.RESIDENT, dtype=torch.int32)]))
    assert bool((tables[0] == -1).all())
    m.hs.close()
    m.mem.close()
