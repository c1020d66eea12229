"""The selective scan's kernels keep every value in registers: a value stored
to scratch where only some lanes are on can come back as something else in the
others, and a reload waits for every load under way.  What the compiler wrote
beside each kernel of the built library says so."""

import re

import pytest


def _spills(blob):
    """{kernel: registers spilled} from the kernels' descriptions, each of which names .symbol before .vgpr_spill_count."""
    out = {}
    name = None
    for m in re.finditer(rb"\.symbol[\xa0-\xbf\xd9\xda].{0,2}?(_Z\w+?)\.kd|\.vgpr_spill_count(.{3})", blob, re.S):
        if m.group(1):
            name = m.group(1).decode()
            continue
        v = m.group(2)   # a small number as it is, larger ones behind 0xcc (8 bits) and 0xcd (16)
        out[name] = v[0] if v[0] < 0x80 else v[1] if v[0] == 0xCC else v[1] << 8 | v[2]
    return out


@pytest.fixture(scope="module")
def spills():
    from tests._libutil import ensure_built

    ensure_built()
    from structured_sparse_state_pdssm_amd._lib import LIB_PATH

    with open(LIB_PATH, "rb") as f:
        return _spills(f.read())


def test_every_layer_kernel_is_described(spills):
    for word, least in (("selscan_kernel", 8), ("selscan_state_kernel", 8), ("selscan_bwd_kernel", 8), ("conv_bwd_kernel", 6), ("norm_bwd_kernel", 8)):
        assert sum(word in k for k in spills) >= least, (word, len(spills))


def test_nothing_is_spilled(spills):
    bad = {k: n for k, n in spills.items() if n and re.search("pdssm_(selscan|conv|norm|ssm)_", k)}
    assert not bad
