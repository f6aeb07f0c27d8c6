"""Which kernels the calls around a batched round launch, on both sides of each rule, checked on the
CPU (the library's host code with the stand-in runtime of ``tests/launch_trace``)."""
import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(__file__), "launch_trace"))
import build_trace  # noqa: E402

SOURCES = ["api.cu", "dq_gemm.cu", "tc_gemm.cu", "gemv.cu", "small_kernels.cu", "moe_kernels.cu", "noalloc.cu",
           "page_assign.cu", "paged_attn.cu", "attn_tc.cu", "attn_tc_bf16.cu", "prefix_attn.cu", "prefix_tc.cu",
           "prefix_tc_bf16.cu", "prefix_own.cu"]


@pytest.fixture(scope="module")
def plan(request):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    patch = pytest.MonkeyPatch()
    patch.setattr(build_trace, "SOURCES", SOURCES)
    patch.setattr(build_trace, "HOST", ["stub_runtime.cpp", "rounds_main.cpp"])
    exe = build_trace.build(out_dir=build_trace.OUT + "_rounds")
    patch.undo()

    def run(command, sms=152):
        _, call = build_trace.run(exe, [f"device {sms} 232448", command])
        assert call["status"] == 0
        return call["launches"]

    return run


def kinds(launches, *names):
    """The launches by which of the names is theirs."""
    return [next(n for n in names if n in launch["name"]) for launch in launches]


SMALL, CLUSTER, PLACE = "page_assign_small", "page_assign_kernel", "page_place"


@pytest.mark.parametrize("B,T,most,maps,want", [
    (48, 17, 1003, 1, [SMALL]), (255, 1, 257, 1, [SMALL]), (255, 1, 258, 1, [CLUSTER, PLACE]),
    (64, 17, 1024, 0, [SMALL]), (64, 17, 1025, 0, [CLUSTER]), (255, 1, 1000, 0, [CLUSTER]),
    (8, 1, 100000, 0, [SMALL]), (8, 320, 100000, 1, [SMALL]), (9, 1, 100000, 0, [CLUSTER]),
    (8, 321, 10, 1, [CLUSTER, PLACE]), (256, 1, 10, 0, [CLUSTER]), (1, 5000, 500, 0, [SMALL]),
])
def test_pages_by_sequences_rows_and_entries(plan, B, T, most, maps, want):
    assert kinds(plan(f"pages {B} {T} {most} {maps}"), SMALL, CLUSTER, PLACE) == want


OWN, PAGED = "prefix_own", "attn_tc_kernel"


def own_form(launches):
    found = [n for launch in launches for n in (OWN, PAGED) if n in launch["name"]]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("B,S,hq,hkv,d,most,want", [
    # heads of 128: one warp, two, four, and several row groups
    (1, 1, 32, 8, 128, 4800, OWN), (1, 1, 32, 8, 128, 4816, PAGED), (4, 1, 32, 8, 128, 9600, OWN),
    (16, 5, 32, 8, 128, 3008, PAGED), (16, 5, 32, 8, 128, 2992, OWN), (16, 16, 32, 8, 128, 992, OWN),
    (16, 16, 32, 8, 128, 1008, PAGED), (4, 32, 32, 8, 128, 992, OWN), (4, 32, 32, 8, 128, 1008, PAGED),
    # heads of 256, one row group: by sequences and heads
    (1, 1, 16, 2, 256, 2400, OWN), (1, 1, 16, 2, 256, 2416, PAGED), (64, 2, 16, 2, 256, 19200, OWN),
    # several row groups: up to half as many as SMs, up to 1.5 an SM, more
    (4, 9, 16, 2, 256, 992, OWN), (4, 9, 16, 2, 256, 1008, PAGED), (16, 9, 16, 2, 256, 496, OWN),
    (16, 9, 16, 2, 256, 512, PAGED), (64, 9, 16, 2, 256, 992, OWN), (64, 9, 16, 2, 256, 1008, PAGED),
])
def test_own_positions_by_rows_sequences_and_tables(plan, B, S, hq, hkv, d, most, want):
    # (a prefix of more positions than few rows take in parts)
    assert own_form(plan(f"prefix {B} {S} {hq} {hkv} {d} 16 1000 {most // 16}")) == want


@pytest.mark.parametrize("B,sms,want", [(7, 152, OWN), (8, 152, PAGED), (8, 160, OWN), (22, 152, PAGED), (23, 152, OWN),
                                         (23, 160, PAGED), (24, 160, OWN)])
def test_row_groups_are_counted_by_the_device(plan, B, sms, want):
    assert own_form(plan(f"prefix {B} 9 16 2 256 16 100 60", sms=sms)) == want
