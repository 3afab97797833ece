"""ISA checks of the MXFP4 and expert kernels (CPU only: hipcc cross-compiles to assembly): nothing
spills, the tiled forms have the LDS and registers for the workgroups per CU that their grids
assume, and the products run on the scaled matrix instructions."""
import os
import re

import pytest

from quantized_prefill_gemm_amd import build as qbuild

pytestmark = pytest.mark.skipif(not os.path.exists(qbuild.hipcc()), reason="hipcc not available")
CSRC = os.path.join(qbuild.HERE, "csrc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    d, out = tmp_path_factory.mktemp("asm"), {}
    for name in ("mxfp4", "mmq_mxfp4", "experts"):
        text = open(qbuild.device_asm(os.path.join(CSRC, name + ".hip"), str(d / (name + ".s")))).read()
        for m in re.finditer(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", text, re.S):
            get = lambda key: int(re.search(key + r" (\d+)", m.group(2)).group(1))  # noqa: E731
            body = text[text.index("\n" + m.group(1) + ":"):]
            out[m.group(1)] = {"lds": get(".amdhsa_group_segment_fixed_size"), "vgpr": get(".amdhsa_next_free_vgpr"),
                               "scratch": get(".amdhsa_private_segment_fixed_size"),
                               "body": body[:body.index("s_endpgm")]}
    return out


def test_nothing_spills(kernels):
    assert len(kernels) > 100
    assert {k: v["scratch"] for k, v in kernels.items() if v["scratch"]} == {}


# template arguments WM, WN, FM, FN, STAGES -> waves, workgroups per CU
TILED = [((2, 2, 1, 1, 3), 4, 2), ((2, 2, 1, 2, 2), 4, 2), ((2, 2, 2, 2, 2), 4, 2), ((2, 4, 4, 2, 2), 8, 1)]


@pytest.mark.parametrize("form,waves,per_cu", TILED)
def test_tiled_forms_fit(kernels, form, waves, per_cu):
    name = "mmq_mxfp4_tiled_kernelI" + "".join(f"Li{v}E" for v in form)
    found = {k: v for k, v in kernels.items() if name in k}
    assert len(found) == 6                                        # three output types, dense and experts
    for k, v in found.items():
        per_simd = 512 // (-(-v["vgpr"] // 8) * 8)
        assert v["lds"] * per_cu <= 163840 and per_simd * 4 // waves >= per_cu, (k, v["lds"], v["vgpr"])


def test_products_use_the_scaled_matrix_instructions(kernels):
    for k, v in kernels.items():
        if "mmq_mxfp4" in k:
            assert "v_mfma_scale_f32_" in v["body"], k
            assert not re.search(r"v_mfma_(?!scale)", v["body"]), k


def test_row_kernels_have_no_wait_between_their_loads(kernels):
    """The weighted sum of 16-byte accesses: the eight loads of four choices' rows follow each
    other with no wait for memory in between."""
    body = next(v["body"] for k, v in kernels.items() if "combine_kernelIDF16bDF16bLi8ELb1E" in k)
    ops = re.findall(r"buffer_load_dwordx4|s_waitcnt[^\n]*vmcnt", body)
    assert "".join("l" if o.startswith("buffer") else "w" for o in ops).find("l" * 8) >= 0
