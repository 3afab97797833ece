"""ISA checks of the kernels over a paged cache (CPU only: hipcc cross-compiles to assembly): nothing spills, the forms
have the LDS and registers for the workgroups per CU that their grids assume, and the loads to LDS, which are inline asm,
keep the wait states that the compiler does not see to there."""
import os
import re

import pytest

from quantized_prefill_gemm_amd import build as qbuild

pytestmark = pytest.mark.skipif(not os.path.exists(qbuild.hipcc()), reason="hipcc not available")
CSRC = os.path.join(qbuild.HERE, "csrc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    d, out = tmp_path_factory.mktemp("asm"), {}
    for name in ("cache_append", "cache_attention"):
        text = open(qbuild.device_asm(os.path.join(CSRC, name + ".hip"), str(d / (name + ".s")))).read()
        for m in re.finditer(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", text, re.S):
            get = lambda key: int(re.search(key + r" (\d+)", m.group(2)).group(1))  # noqa: E731
            body = text[text.index("\n" + m.group(1) + ":"):]
            lines = [x.strip() for x in body[:body.index("s_endpgm")].split("\n")]
            out[m.group(1)] = {"lds": get(".amdhsa_group_segment_fixed_size"), "vgpr": get(".amdhsa_next_free_vgpr"),
                               "scratch": get(".amdhsa_private_segment_fixed_size"),
                               "body": [x for x in lines if x and x[0] not in ";." and not x.endswith(":")]}
    return out


def test_nothing_spills(kernels):
    assert len(kernels) > 50
    assert {k: v["scratch"] for k, v in kernels.items() if v["scratch"]} == {}


# template arguments DP, WC, WK, KT -> waves, workgroups per CU
FORMS = [((64, 4, 1, 64), 4, 2), ((128, 4, 1, 64), 4, 2), ((64, 4, 2, 64), 8, 1), ((128, 4, 2, 64), 8, 1), ((64, 2, 4, 32), 8, 1),
         ((128, 2, 4, 32), 8, 1), ((64, 1, 4, 32), 4, 2), ((128, 1, 4, 32), 4, 1), ((256, 4, 1, 32), 4, 1), ((256, 2, 2, 32), 4, 1),
         ((256, 1, 2, 32), 2, 1)]


@pytest.mark.parametrize("form,waves,per_cu", FORMS)
def test_forms_fit(kernels, form, waves, per_cu):
    name = "".join(f"Li{v}E" for v in form)
    found = {k: v for k, v in kernels.items() if "cache_attention_kernel" in k and name in k}
    assert len(found) == 4                                        # two cache types, one and more pieces of a share
    for k, v in found.items():
        per_simd = min(512 // (-(-v["vgpr"] // 8) * 8), 8)
        assert v["lds"] * per_cu <= 163840 and per_simd * 4 // waves >= per_cu, (k, v["lds"], v["vgpr"])


def test_loads_to_lds_wait_for_their_scalars(kernels):
    """Five wait states from a scalar written by the VALU (v_readlane, v_readfirstlane) to the load that has it in its
    descriptor, and one from a write of m0."""
    loads = 0
    for k, v in kernels.items():
        body = v["body"]
        for i, x in enumerate(body):
            if not (x.startswith("buffer_load") and x.endswith(" lds")):
                continue
            loads += 1
            lo, hi = map(int, re.search(r"s\[(\d+):(\d+)\]", x).groups())
            states = 0
            for y in reversed(body[max(0, i - 12):i]):
                if states >= 5:
                    break
                m = re.match(r"v_read(?:first)?lane_b32 s(\d+)", y)
                assert not (m and lo <= int(m.group(1)) <= hi), (k, y, x, states)
                assert not (states < 1 and re.match(r"s_\w+ m0,", y)), (k, y, x)
                states += int(y.split()[1]) + 1 if y.startswith("s_nop") else 1
    assert loads > 400


def test_no_wait_for_the_stage_under_way(kernels):
    """Between the barrier of a round and its first product, nothing of the compiler's waits for vector memory in the
    short way: the stage that has just been asked for is under way there."""
    for k, v in kernels.items():
        if "cache_attention_kernel" not in k:
            continue
        body = v["body"]
        at = max(i for i, x in enumerate(body) if x.startswith("buffer_load") and x.endswith(" lds"))
        upto = next(i for i in range(at, len(body)) if "mfma" in body[i])
        assert not any("vmcnt" in x for x in body[at:upto]), k


@pytest.fixture(scope="module")
def whole(kernels, tmp_path_factory):
    """The attention kernels to their last instruction (a walk may lie behind the first s_endpgm)."""
    path = next(p for p in sorted(tmp_path_factory.getbasetemp().glob("asm*/cache_attention.s")))
    text, out = path.read_text(), {}
    for name in kernels:
        if "cache_attention_kernel" in name:
            body = text[text.index("\n" + name + ":"):text.index(".amdhsa_kernel " + name)]
            lines = [x.strip() for x in body.split("\n")]
            out[name] = [x for x in lines if x and x[0] not in ";." and not x.endswith(":")]
    return out


def is_load(x):
    return x.startswith("buffer_load") and x.endswith(" lds")


def test_loads_of_both_walks_wait_for_their_scalars(whole):
    """As above, to the last load of a kernel."""
    loads = 0
    for k, body in whole.items():
        for i, x in enumerate(body):
            if not is_load(x):
                continue
            loads += 1
            lo, hi = map(int, re.search(r"s\[(\d+):(\d+)\]", x).groups())
            states = 0
            for y in reversed(body[max(0, i - 12):i]):
                if states >= 5:
                    break
                m = re.match(r"v_read(?:first)?lane_b32 s(\d+)", y)
                assert not (m and lo <= int(m.group(1)) <= hi), (k, y, x, states)
                assert not (states < 1 and re.match(r"s_\w+ m0,", y)), (k, y, x)
                states += int(y.split()[1]) + 1 if y.startswith("s_nop") else 1
    assert loads > 1000


def test_no_wait_for_the_stage_under_way_in_either_walk(whole):
    """From a round's last load to its first product nothing waits for vector memory, once in each walk. (Behind the loads
    of the first stage, before the loop, the queries are waited for.)"""
    for k, body in whole.items():
        walks, under_way = 0, False
        for x in body:
            if is_load(x):
                under_way = True
            elif x.startswith("s_waitcnt") and "vmcnt" in x:
                under_way = False
            elif "mfma" in x and under_way:
                walks, under_way = walks + 1, False
        assert walks == 2, (k, walks)
