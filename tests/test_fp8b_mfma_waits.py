"""The wait states behind the matrix instructions of the block-scaled fp8 products and of the gradient of a weight, read
from the disassembly of the built library with the scan of test_mfma_waits."""
import pytest

import precision_quantized_linear_amd as qpl
import test_mfma_waits as scan

# passes + 4, as there; both instructions take eight passes
WAITS = {"v_mfma_scale_f32_16x16x128_f8f6f4": 12, "v_mfma_f32_32x32x16_bf16": 12}


@pytest.fixture
def waits(monkeypatch):
    for op, n in WAITS.items():
        monkeypatch.setitem(scan.WAITS, op, n)


@pytest.mark.parametrize("behind,found", [("s_nop 7", 1), ("s_nop 10", 1), ("s_nop 11", 0)])
def test_the_scan_knows_the_instructions(waits, behind, found):
    text = f"""
  v_mfma_scale_f32_16x16x128_f8f6f4 v[4:7], v[8:15], v[16:23], 0, v40, v40 op_sel_hi:[0,0,0]
  {behind}
  v_fma_f32 v30, v4, v31, v30
  s_endpgm
"""
    assert len(scan.early_reads(scan.listing(text))) == found


@pytest.mark.skipif(scan.OBJDUMP is None, reason="no llvm-objdump")
@pytest.mark.parametrize("match,least", [("k_fp8b_", 20), ("k_weight_grad", 2)])
def test_no_reader_stands_too_close(waits, match, least):
    found = scan.kernels(scan.code_objects(qpl.LIB_PATH), match)
    ops = {n: {t.split()[0] for _, t, _ in ins if "mfma" in t.split()[0]} for n, ins in found.items()}
    assert sum(bool(v) for v in ops.values()) >= least and set().union(*ops.values()) <= set(WAITS)
    bad = {n: scan.early_reads(ins)[:3] for n, ins in found.items() if scan.early_reads(ins)}
    assert not bad
