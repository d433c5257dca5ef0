"""Loads into LDS of the block-scaled fp8 products and of the gradient of a weight, read from the disassembly of the
built library: no part of an address stands in the scalar offset, so what a lane's own offset and the descriptor's start
and size say is all that decides whether it reads memory or gets zeros."""
import re

import pytest

import precision_quantized_linear_amd as qpl
import test_mfma_waits as scan

LOAD = re.compile(r"^buffer_load_\S+ v\d+, s\[\d+:\d+\], (\S+) .*\blds\b")


@pytest.mark.parametrize("line,offset", [("buffer_load_dwordx4 v5, s[8:11], 0 offen lds", "0"),
                                         ("buffer_load_dwordx4 v5, s[8:11], s20 offen lds", "s20"),
                                         ("buffer_load_dword v117, s[8:11], 0 offen lds", "0")])
def test_the_scan_reads_the_scalar_offset(line, offset):
    assert LOAD.match(line).group(1) == offset


@pytest.mark.skipif(scan.OBJDUMP is None, reason="no llvm-objdump")
@pytest.mark.parametrize("match,least", [("k_fp8b_staged", 18), ("k_weight_grad", 2)])
def test_no_load_into_lds_has_a_scalar_offset(match, least):
    found = scan.kernels(scan.code_objects(qpl.LIB_PATH), match)
    loads = {n: [t for _, t, _ in ins if t.startswith("buffer_load") and t.endswith("lds")] for n, ins in found.items()}
    assert sum(bool(v) for v in loads.values()) >= least
    assert not {n: v[:3] for n, v in loads.items() if any(LOAD.match(t).group(1) != "0" for t in v)}
