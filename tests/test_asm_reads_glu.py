"""The check of test_asm_reads.py on the gated products' instantiations of the same kernel
(csrc/gemm_glu.hip): no register of an outstanding transposing read is touched."""
import os
import subprocess

import pytest

from test_asm_reads import early_touches, kernels_with_tr_reads


def test_no_register_of_an_outstanding_transposing_read_is_touched(tmp_path):
    from tensor_transformer_mlp_03_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path / "gemm_glu.s"
    cmd = [cc, *build.CFLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "gemm_glu.hip"), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    kernels = kernels_with_tr_reads(out.read_text())
    assert len(kernels) >= 12, "the N-contiguous kernels of three tiles and four activations issue transposing reads"
    bad = {k: early_touches(b) for k, b in kernels.items()}
    assert not any(bad.values()), {k: v[:3] for k, v in bad.items() if v}


def test_nor_by_the_products_in_one_launch(tmp_path):
    """The same of gemm_group.hip, whose group kernels hold the body for both layouts."""
    from tensor_transformer_mlp_03_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path / "gemm_group.s"
    cmd = [cc, *build.CFLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "gemm_group.hip"), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    kernels = kernels_with_tr_reads(out.read_text())
    assert len(kernels) >= 4, "one for each pair of output types"
    bad = {k: early_touches(b) for k, b in kernels.items()}
    assert not any(bad.values()), {k: v[:3] for k, v in bad.items() if v}
