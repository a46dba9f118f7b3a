"""CPU test of the rule that says how many threads pick a row's cut or token
(``picker_threads``), built for the host with g++: whatever it chooses, the
work-group's arrays hold the row's pieces and its threads look at all of them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_cross_entropy_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is needed")
    exe = str(tmp_path_factory.mktemp("picker") / "picker_host")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "host", "picker_host.cpp"), "-o", exe], check=True, capture_output=True)

    def run(cases):
        text = "".join(f"{n} {v} {int(a)}\n" for n, v, a in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [tuple(map(int, out[3 * i:3 * i + 3])) for i in range(len(cases))]
    return run


def test_a_rows_pieces_always_fit(rule):
    sizes = sorted({v for e in range(11, 25) for v in ((1 << e) - 1, 1 << e, (1 << e) + 1) if v <= 1 << 24}
                   | {k * 8192 + d for k in range(1, 2048, 7) for d in (0, 1)} | {202048, 129279, 1 << 24})
    cases = [(n, v, a) for v in sizes for n in (1, 256, 257, 4096, 1 << 21) for a in (False, True)]
    for case, (threads, pieces, room) in zip(cases, rule(cases)):
        assert threads in (512, 1024) and pieces <= room and room <= 2 * threads, case


def test_where_two_rows_share_a_compute_unit(rule):
    for case, threads in [((256, 4000, True), 1024), ((257, 4000, False), 512), ((257, 65536, False), 512),
                          ((257, 65537, False), 1024), ((257, 65537, True), 512), ((480, 202048, True), 512),
                          ((480, 202048, False), 1024), ((257, 2097152, True), 512), ((257, 2097153, True), 1024),
                          ((257, 1 << 24, True), 1024), ((1 << 12, 1 << 24, True), 1024)]:
        assert rule([case])[0][0] == threads, case
