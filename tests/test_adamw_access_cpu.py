"""The AdamW step's choice between vectors and single elements, compiled for the
host: whatever the addresses of a tensor's arrays, every access of the chosen
path is aligned to its own width."""
import itertools
import os
import shutil
import subprocess

import pytest

import mixture_experts_layer_logit_b200 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_logit_b200", "csrc")
SRC = os.path.join(ROOT, "tests", "adamw_access_check.cpp")
F32, BF16, F16 = moe.MOE_DTYPE_F32, moe.MOE_DTYPE_BF16, moe.MOE_DTYPE_F16
BASE = 1 << 20
OPERANDS = ("param", "grad", "master", "m", "v")


def size(dt):
    return 4 if dt == F32 else 2


def widest(vectors, bits, p, g):
    """Bytes of the widest access to each operand on a path of the kernel, in the order of OPERANDS."""
    lane = lambda dt: 8 * size(dt)   # noqa: E731
    if not vectors:
        return size(p), size(g), 4, bits // 8, bits // 8
    if bits == 8:   # copies of 16 bytes in, eight elements or codes of a lane out
        return lane(p), 16, 32, 16, 16
    return lane(p), lane(g), 32, 32, 32


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("access") / "adamw_access_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), SRC, "-o", exe],
                   check=True)

    def run(rows):
        text = "\n".join(" ".join(str(x) for x in r) for r in rows)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.split()
        assert len(out) == len(rows)
        return [int(x) for x in out]
    return run


def shifts(dt_bytes):
    return [i for i in (0, 1, 2, 4, 8, 12, 16, 24, 32, 48) if i % dt_bytes == 0]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("p", [F32, BF16, F16])
@pytest.mark.parametrize("g", [F32, BF16, F16])
@pytest.mark.parametrize("master", [False, True])
def test_every_access_is_aligned(choose, bits, p, g, master):
    per = [shifts(size(p)), shifts(size(g)), shifts(4) if master else [None], shifts(bits // 8), shifts(bits // 8)]
    rows = [(bits, p, g, *(0 if s is None else BASE + s for s in at)) for at in itertools.product(*per)]
    for row, vectors in zip(rows, choose(rows)):
        for name, at, width in zip(OPERANDS, row[3:], widest(vectors, bits, p, g)):
            assert at % width == 0, (name, at - BASE, width, row)
    assert choose([(bits, p, g, BASE, BASE, BASE if master else 0, BASE, BASE)]) == [1]


@pytest.mark.parametrize("bits,g,shift,vectors", [(32, F32, 16, 0), (32, F32, 32, 1), (32, BF16, 16, 1), (32, BF16, 8, 0),
                                                  (8, F32, 16, 1), (8, F32, 8, 0), (8, BF16, 16, 1)])
def test_gradients_cut_from_a_flat_buffer(choose, bits, g, shift, vectors):
    assert choose([(bits, BF16, g, BASE, BASE + shift, BASE, BASE, BASE)]) == [vectors]
