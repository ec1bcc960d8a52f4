"""Checks on the compiled kernels of the dense path (gfx950 assembly, built here
with hipcc).

* No kernel of the product spills in its K loop, and only one has scratch at all (the widest
  tile with scales of b's rows: addresses that its loop does not touch).
* The K loop of the E4M3 product is one block of code without a full drain of
  the direct global->LDS loads (``s_waitcnt vmcnt(0)``) but the one that tiles
  with two rounds in LDS wait at for the next: another would come from a vector
  load of scales, or from a read of a stage through a type that the compiler
  cannot tell apart from what the direct loads write, and would serialise the
  loads without changing any result.
"""

import os
import re
import subprocess
import tempfile

import pytest

from fp8_mixture_experts_amd import build as BLD

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixture_experts_amd", "csrc")


def _kernels(source):
    """name -> (lines of its code, bytes of scratch)."""
    if not os.path.exists(BLD.HIPCC):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "x.s")
        cmd = [BLD.HIPCC, "-x", "hip", *BLD.COMMON, *BLD.DEVICE_ONLY, "--offload-device-only", "-S", os.path.join(CSRC, source), "-o", out]
        r = subprocess.run([c for c in cmd if c != "-fPIC"], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        text = open(out).read()
    scratch = {}
    for chunk in text[text.index("amdhsa.kernels:"):].split("\n  - ")[1:]:
        name = re.search(r"\.name:\s+(_Z\S+)", chunk)
        if name:
            scratch[name.group(1)] = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", chunk).group(1))
    code = {}
    for name in scratch:
        start = re.search(r"^" + re.escape(name) + ":", text, re.M).start()
        code[name] = text[start:text.index(".Lfunc_end", start)].split("\n")
    return {n: (code[n], scratch[n]) for n in scratch}


def _blocks(lines):
    """The code between one label and the next."""
    at = [i for i, line in enumerate(lines) if re.match(r"\.LBB\d+_\d+:", line)]
    return [lines[i:j] for i, j in zip([0] + at, at + [len(lines)])]


def _k_loop(lines):
    blocks = [b for b in _blocks(lines) if any("v_mfma" in line for line in b)]
    assert len(blocks) == 1, len(blocks)
    # up to the branch that goes on with the loop: behind it is its exit
    return blocks[0][:max(i for i, line in enumerate(blocks[0]) if "s_cbranch" in line) + 1]


@pytest.fixture(scope="module")
def product():
    return _kernels("product.hip")


def _tile(name):
    return [int(v) for v in re.findall(r"Li(\d+)E", name)[:6]] if "Tile" in name else None


def test_product_s_loops_do_not_spill(product):
    assert len([n for n in product if _tile(n)]) == 28
    for name, (lines, scratch) in product.items():
        widest_by_rows = _tile(name) and _tile(name)[:2] == [256, 256] and "ELb0ELb1E" in name
        assert scratch == 0 or (widest_by_rows and scratch <= 128), name
        if _tile(name):
            assert not any("scratch_" in line for line in _k_loop(lines)), name


def test_product_s_k_loop_is_one_block_that_keeps_loads_in_flight(product):
    for name, (lines, _) in product.items():
        tile = _tile(name)
        if not tile:
            continue
        loop = _k_loop(lines)
        count = sum("v_mfma" in line for line in loop)
        bm, bn, wm, wn, _, stages = tile
        exact = "ELb1ELb" in name
        assert count == bm // wm // 16 * (bn // wn // 16) * (4 if exact else 1), (name, count)
        drains = sum(bool(re.search(r"s_waitcnt.*vmcnt\(0\)", line)) for line in loop)
        early = (bm, bn) == (256, 256)
        assert drains <= (1 if stages == 2 and not early else 0), (name, drains)


@pytest.mark.parametrize("source", ["quantize.hip", "rotary.hip"])
def test_the_other_kernels_have_no_scratch(source):
    kernels = _kernels(source)
    assert kernels
    for name, (_, scratch) in kernels.items():
        assert scratch == 0, name
