"""Static checks of the compiled E4M3 product, weight gradient and norm kernels (CPU
only): LDS written by one lane and read by another of the same wave has a barrier
between, and 16-bit results are fp32 values first."""
import os
import re
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import asm_hazards as H  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_mxgemm_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which(os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")) is None,
                                reason="hipcc not found")


@pytest.fixture(scope="module")
def asm():
    from block_scaled_precision_mxgemm_amd import build as B
    return {f: H.compile_to_asm(os.path.join(CSRC, f + ".hip"), B.FLAGS, B.HIPCC)
            for f in ("gemm_fp8", "fp8_weight_grad", "rmsnorm")}


def unordered(body):
    """(runs of reads behind a barrier, reads straight behind writes)"""
    last, runs, bad = "", 0, 0
    for op in re.findall(r"^\s*(?:(ds_write|ds_read_b128|s_barrier)|(; wave barrier))", body, re.M):
        op = op[0] or op[1]
        bad += last == "ds_write" and op == "ds_read_b128"
        runs += last in ("; wave barrier", "s_barrier") and op == "ds_read_b128"
        last = op
    return runs, bad


def test_the_check_sees_a_missing_barrier():
    write, read = "\tds_write_b64 v1, v[2:3]\n", "\tds_read_b128 v[4:7], v1\n"
    assert unordered(write + read) == (0, 1)
    assert unordered(write + "\t; wave barrier\n" + read) == (1, 0)
    assert unordered(write + "\ts_barrier\n" + read + read) == (1, 0)


@pytest.mark.parametrize("source,kernel,count", [("gemm_fp8", "fp8_ring_kernel", 10), ("fp8_weight_grad", "fp8_weight_grad_kernel", 12)])
def test_output_steps_keep_their_lds_order(asm, source, kernel, count):
    seen = 0
    for m in re.finditer(r"^(_ZN\S*%s\S*):" % kernel, asm[source], re.M):
        runs, bad = unordered(asm[source][m.end():asm[source].index(".Lfunc_end", m.end())])
        assert bad == 0 and runs >= 4, (m.group(1), runs, bad)
        seen += 1
    assert seen == count


def test_16_bit_results_are_rounded_to_fp32_first(asm):
    """No conversion to fp16 is joined with the operation before it (one rounding
    instead of two)."""
    for source, text in asm.items():
        assert "v_cvt_f16_f32" in text or "v_cvt_pk" in text
        assert not re.search(r"v_(fma|mad)_mix(lo|hi)", text), source
